"""The gated delta rule on the GPU against its token-by-token definition in 64 bits."""
import ctypes

import pytest
import torch

import device_wide_prefix_amd as dws
from delta_reference import close, inputs, reference, tolerance
from gpu_util import note

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
NAMES = ("q", "k", "v", "g", "beta")


def forward(x, offsets, initial, scale=None, **more):
    out = dws.delta_rule(*(x[a] for a in NAMES), offsets=offsets, initial_state=initial, scale=scale, **more)
    torch.cuda.synchronize()
    return out


def gradients(x, offsets, initial, scale, d_out, d_final):
    """The reference's gradients, by differentiating it."""
    leaves = {a: x[a].double().cpu().requires_grad_() for a in NAMES if x[a] is not None}
    s = None if initial is None else initial.double().cpu().requires_grad_()
    o, f = reference(leaves["q"], leaves["k"], leaves["v"], leaves.get("g"), leaves["beta"], offsets.tolist(), s, scale)
    loss = (o * d_out.double().cpu()).sum()
    if d_final is not None:
        loss = loss + (f * d_final.double().cpu()).sum()
    wanted = [leaves[a] for a in NAMES if a in leaves] + ([s] if s is not None else [])
    got = list(torch.autograd.grad(loss, wanted, allow_unused=True))
    got = [torch.zeros_like(w) if y is None else y for y, w in zip(got, wanted)]
    if "g" not in leaves:
        got.insert(3, None)
    return got + ([None] if s is None else [])


# lens, heads_qk, heads_v, dim_k, dim_v, initial state
SHAPES = [
    ([1], 1, 1, 1, 1, True),
    ([31], 1, 1, 64, 64, False),
    ([32], 1, 2, 64, 16, True),
    ([33, 1, 0, 2], 1, 1, 8, 8, True),
    ([63, 64, 65], 2, 2, 64, 64, False),
    ([0, 129, 0], 2, 6, 40, 24, True),
    ([127, 128], 1, 1, 65, 17, True),
    ([200], 1, 1, 128, 128, True),
    ([97, 70], 3, 3, 100, 130, False),
    ([130], 1, 2, 256, 256, True),
    ([70, 3], 1, 1, 129, 255, True),
]


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("lens,hk,hv,dk,dv,init", SHAPES)
def test_forward(gpu, lens, hk, hv, dk, dv, init, dtype):
    note(f"delta forward {lens} {hk} {hv} {dk} {dv} {init} {dtype}")
    x, offsets, initial = inputs(1, lens, hk, hv, dk, dv, dtype, init=init)
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), None if initial is None else initial.double().cpu(), dk ** -0.5)
    close(forward(x, offsets, initial), want, dtype, "out")
    out, state = forward(x, offsets, initial, final_state=True)
    close(out, want, dtype, "out")
    close(state, final, dtype, "state")


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("lens,hk,hv,dk,dv,init", SHAPES)
def test_backward(gpu, lens, hk, hv, dk, dv, init, dtype):
    note(f"delta backward {lens} {hk} {hv} {dk} {dv} {init} {dtype}")
    x, offsets, initial = inputs(2, lens, hk, hv, dk, dv, dtype, init=init)
    gen = torch.Generator().manual_seed(3)
    d_out = torch.randn(x["v"].shape, generator=gen).to(dtype).cuda()
    d_final = 0.3 * torch.randn(len(lens), hv, dk, dv, generator=gen).cuda() if init else None
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial, d_final_state=d_final)
    torch.cuda.synchronize()
    want = gradients(x, offsets, initial, dk ** -0.5, d_out, d_final)
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
        assert (a is None) == (b is None)
        if a is not None:
            assert a.dtype == dtype
            close(a, b, dtype, what)


# sequences and heads enough for workgroups of the widest kind on every compute unit
MANY = [([0, 70, 33, 1, 64, 5] * 6, 8, 8, 64, 64), ([65, 2, 40, 129] * 9, 2, 8, 128, 70), ([33, 64, 31] * 9, 3, 12, 200, 40),
        ([20, 90] * 17, 8, 8, 256, 17), ([30] * 65, 2, 4, 128, 128)]


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", MANY)
def test_many_sequences(gpu, lens, hk, hv, dk, dv, dtype):
    note(f"delta many {len(lens)} {hk} {hv} {dk} {dv} {dtype}")
    assert len(lens) * hv * -(-dv // 64) >= 256
    x, offsets, initial = inputs(21, lens, hk, hv, dk, dv, dtype, tail=3)
    ends = offsets.tolist()
    some = sorted({0, 1, 2, 3, len(lens) // 2, len(lens) - 2, len(lens) - 1})
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    d_final = 0.3 * torch.randn(initial.shape, generator=torch.Generator().manual_seed(4)).cuda()
    out, state = forward(x, offsets, initial, final_state=True)
    plain = forward(x, offsets, initial)
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial, d_final_state=d_final)
    assert (out[ends[-1]:] == 0).all() and (got[0][ends[-1]:] == 0).all()
    for i in some:
        rows = slice(ends[i], ends[i + 1])
        y = {a: x[a][rows] for a in NAMES}
        at = torch.tensor([0, lens[i]])
        want, final = reference(*(y[a] for a in NAMES), at.tolist(), initial[i: i + 1].double().cpu(), dk ** -0.5)
        close(out[rows], want, dtype, "out")
        close(plain[rows], want, dtype, "out")
        close(state[i: i + 1], final, dtype, "state")
        want = gradients(y, at, initial[i: i + 1], dk ** -0.5, d_out[rows], d_final[i: i + 1])
        for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
            close(a[rows] if what != "d_initial" else a[i: i + 1], b, dtype, what, f"{i}")


@pytest.mark.parametrize("gates", [(FP32, FP32), (BF16, BF16), (FP16, FP32), (FP32, FP16)])
def test_gate_types(gpu, gates):
    x, offsets, initial = inputs(4, [70, 40], 1, 2, 64, 32, BF16, gates=gates)
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), initial.double().cpu(), 0.5)
    out, state = forward(x, offsets, initial, scale=0.5, final_state=True)
    close(out, want, BF16, "out")
    close(state, final, BF16, "state")
    pool = initial.clone()
    close(dws.delta_rule_step(*(x[a] for a in NAMES), pool, offsets=offsets, scale=0.5), want, BF16, "out")
    close(pool, final, FP32, "state")


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_no_decay(gpu, dtype):
    x, offsets, initial = inputs(5, [150], 1, 1, 64, 48, dtype)
    x["g"] = None
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), initial.double().cpu(), 0.125)
    out, state = forward(x, offsets, initial, final_state=True)
    close(out, want, dtype, "out")
    close(state, final, dtype, "state")
    d_out = torch.ones_like(x["v"])
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
    want = gradients(x, offsets, initial, 0.125, d_out, None)
    assert got[3] is None
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
        if a is not None:
            close(a, b, dtype, what)


def special(kind, dtype, n=140, hv=2, dk=64, dv=32):
    x, offsets, initial = inputs(6, [n], 1, hv, dk, dv, dtype)
    if kind == "forget":                 # -infinity, and more than any sum of 64 decays
        x["g"][5] = -float("inf")
        x["g"][70:75] = -float("inf")
        x["g"][20, 0] = -200.0
        x["g"][100:, 1] = -1e30
        x["g"][n - 1] = torch.finfo(FP32).min
    elif kind == "long_decay":           # sums of hundreds whose differences are small
        x["g"][:] = -60.0
        x["g"][::3] = -1e-3
    elif kind == "beta_zero":            # tokens that change nothing
        x["beta"][::2] = 0
        x["beta"][64:128] = 0
    elif kind == "same_keys":            # every key alike: the system's powers grow, its inverse does not
        x["k"][:] = x["k"][:1]
        x["beta"][:] = 1
        x["g"][:] = 0
    elif kind == "growth":
        x["g"][:] = 0.01
    return x, offsets, initial


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("kind", ["forget", "long_decay", "beta_zero", "same_keys", "growth"])
def test_special_gates(gpu, kind, dtype):
    note(f"delta special {kind} {dtype}")
    x, offsets, initial = special(kind, dtype)
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), initial.double().cpu(), 0.125)
    out, state = forward(x, offsets, initial, final_state=True)
    close(out, want, dtype, "out", kind)
    close(state, final, dtype, "state", kind)
    pool = initial.clone()
    close(dws.delta_rule_step(*(x[a] for a in NAMES), pool, scale=0.125), want, dtype, "out", kind)
    close(pool, final, FP32, "state", kind)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), initial_state=initial, scale=0.125)
    if kind == "forget":                 # exp's derivative at -infinity is 0, which autograd's 0 * inf is not
        x["g"] = x["g"].clamp(min=-1e4)
    want = gradients(x, offsets, initial, 0.125, d_out, None)
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
        close(a, b, dtype, what, kind)


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("lens,dk,dv", [([42, 6, 21, 14, 28, 126, 54, 8, 2, 11, 130, 94], 256, 128), ([66, 111, 28, 27, 146], 128, 104),
                                        ([47, 189], 200, 96)])
def test_gradients_are_near_their_own_rounding(gpu, lens, dk, dv, dtype):
    """Beside the result's rounding, at most one of the same size on the way (an operand in one part), independent of it:
    sqrt(2) times it, and a fifth more for sums that cancel in part."""
    x, offsets, initial = inputs(27, lens, 1, 2, dk, dv, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
    want = gradients(x, offsets, initial, dk ** -0.5, d_out, None)
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
        off, rounding = (a.double().cpu() - b).norm(), (b.to(dtype).double() - b).norm()
        assert off <= 1.2 * 2 ** 0.5 * rounding, f"{what}: off by {off / rounding:.2f} times its rounding"


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_gradient_against_differences(gpu, dtype):
    """The kernel's gradients along a direction against a central difference of the 64-bit definition. The difference's
    own error is h^2 / 6 of the third derivative: below 1e-6 of it for h = 1e-3 at these sizes."""
    x, offsets, initial = inputs(7, [75, 30], 1, 2, 32, 16, dtype)
    gen = torch.Generator().manual_seed(8)
    d_out = torch.randn(x["v"].shape, generator=gen).to(dtype).cuda()
    d_final = torch.randn(initial.shape, generator=gen).cuda()
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial, d_final_state=d_final)
    base = {a: x[a].double().cpu() for a in NAMES}
    base["s"] = initial.double().cpu()

    def loss(y):
        o, f = reference(*(y[a] for a in NAMES), offsets.tolist(), y["s"], 32 ** -0.5)
        return ((o * d_out.double().cpu()).sum() + (f * d_final.double().cpu()).sum()).item()

    h = 1e-3
    for a, d in zip(NAMES + ("s",), got):
        way = torch.randn(base[a].shape, generator=gen, dtype=torch.float64)
        slope = (loss({**base, a: base[a] + h * way}) - loss({**base, a: base[a] - h * way})) / (2 * h)
        mine = (d.double().cpu() * way).sum().item()
        # an error of tolerance() of the gradient's norm, along a direction of norm sqrt(n) that knows nothing of it,
        # five deviations far
        allowed = 5 * tolerance(dtype, "d" + a) * d.double().norm().item() + 1e-5 * abs(slope) + 1e-6
        assert abs(mine - slope) <= allowed, (a, mine, slope, allowed)


@pytest.mark.parametrize("dtype", [FP32, BF16])
def test_strides(gpu, dtype):
    """Parts of one buffer, one element off 16-byte alignment, heads outermost, and repeated rows and heads."""
    lens, hk, hv, dk, dv = [70, 33], 2, 4, 48, 40
    x, offsets, initial = inputs(9, lens, hk, hv, dk, dv, dtype)
    n = sum(lens)
    plain = forward(x, offsets, initial)
    d_out = torch.randn(n, hv, dv, generator=torch.Generator().manual_seed(2)).to(dtype).cuda()
    plain_grads = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
    for shift in (0, 1):
        fused = torch.zeros(n, 2 * hk * dk + hv * dv + 16 + shift, dtype=dtype, device="cuda")
        y = dict(x)
        at = shift
        for a, h, d in (("q", hk, dk), ("k", hk, dk), ("v", hv, dv)):
            y[a] = fused[:, at: at + h * d].unflatten(1, (h, d))
            y[a].copy_(x[a])
            at += h * d
        for a in ("g", "beta"):
            y[a] = x[a].t().contiguous().t()
        assert torch.equal(forward(y, offsets, initial), plain)
        d_view = torch.zeros(hv, n, dv + 3, dtype=dtype, device="cuda")[:, :, shift: shift + dv].transpose(0, 1)
        d_view.copy_(d_out)
        got = dws.delta_rule_backward(d_view, *(y[a] for a in NAMES), offsets=offsets, initial_state=initial)
        for a, b in zip(got, plain_grads):
            assert torch.equal(a, b)
    y = {a: (x[a].transpose(0, 1).contiguous().transpose(0, 1) if x[a].dim() == 3 else x[a]) for a in NAMES}
    out = torch.full((hv, n, dv), 7.0, dtype=dtype, device="cuda").transpose(0, 1)
    assert forward(y, offsets, initial, out=out) is out
    assert torch.equal(out, plain)
    pool = initial.clone()
    dws.delta_rule_step(*(y[a] for a in NAMES), pool, offsets=offsets, out=out)
    close(out, plain, dtype, "dg")      # two results of the type, each off by its own tolerance
    # one query and key for all heads and one v for all tokens, by strides of 0
    y = dict(x)
    y["q"], y["k"] = x["q"][:, :1].expand(n, hk, dk), x["k"][:, :1].expand(n, hk, dk)
    y["v"] = x["v"][:1].expand(n, hv, dv)
    whole = {a: b.contiguous() for a, b in y.items()}
    assert torch.equal(forward(y, offsets, initial), forward(whole, offsets, initial))


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("tail", [1, 53, 130])
def test_rows_behind_the_last_sequence(gpu, dtype, tail):
    """They are not read, and stay as they were in a given output; in a new one, and in gradients, they are 0."""
    x, offsets, initial = inputs(10, [10], 1, 2, 32, 24, dtype, tail=tail)
    for a in NAMES:
        x[a][10:] = float("nan")
    want, final = reference(*(x[a][:10] for a in NAMES), [0, 10], initial.double().cpu(), 32 ** -0.5)
    out = torch.full(x["v"].shape, 5.0, dtype=dtype, device="cuda")
    _, state = forward(x, offsets, initial, out=out, final_state=True)
    close(out[:10], want, dtype, "out")
    close(state, final, dtype, "state")
    assert (out[10:] == 5).all()
    assert (forward(x, offsets, initial)[10:] == 0).all()
    d_out = torch.full(x["v"].shape, float("nan"), dtype=dtype, device="cuda")
    d_out[:10] = 1
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
    for a in got[:5]:
        assert torch.isfinite(a).all() and (a[10:] == 0).all()
    out.fill_(5)
    pool = initial.clone()
    dws.delta_rule_step(*(x[a] for a in NAMES), pool, offsets=offsets, out=out)
    close(out[:10], want, dtype, "out")
    assert (out[10:] == 5).all()


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("head,lens,tail", [(1, [10], 0), (65, [10, 70], 3), (200, [0], 0), (130, [3, 0], 70)])
def test_rows_before_the_first_sequence(gpu, dtype, head, lens, tail):
    """As those behind the last one."""
    x, offsets, initial = inputs(23, lens, 1, 2, 32, 24, dtype, tail=head + tail)
    offsets += head
    end = head + sum(lens)
    for a in NAMES:
        x[a][:head] = x[a][end:] = float("nan")
    want, final = reference(*(x[a][head:end] for a in NAMES), [i - head for i in offsets.tolist()], initial.double().cpu(), 32 ** -0.5)
    out = torch.full(x["v"].shape, 5.0, dtype=dtype, device="cuda")
    _, state = forward(x, offsets, initial, out=out, final_state=True)
    close(out[head:end], want, dtype, "out")
    close(state, final, dtype, "state")
    assert (out[:head] == 5).all() and (out[end:] == 5).all()

    def rest_is_zero(a):
        return torch.isfinite(a).all() and (a[:head] == 0).all() and (a[end:] == 0).all()

    dirty = [torch.full_like(x[a], float("nan")) for a in NAMES]      # what new tensors find in their memory
    del dirty
    assert rest_is_zero(forward(x, offsets, initial))
    d_out = torch.full(x["v"].shape, float("nan"), dtype=dtype, device="cuda")
    d_out[head:end] = 1
    dirty = [torch.full_like(x[a], float("nan")) for a in NAMES]
    del dirty
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
    assert all(rest_is_zero(a) for a in got[:5])


@pytest.mark.parametrize("dtype", [FP32, BF16])
@pytest.mark.parametrize("what", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("value", ["nan", "inf"])
def test_what_is_not_finite_stays_in_its_sequence_and_head(gpu, dtype, what, value):
    """One bad element of one head: other sequences, heads and earlier chunks give the same bits."""
    lens, at = [200, 70, 130], 200 + 69          # the second sequence's last token but one
    x, offsets, initial = inputs(24, lens + [64], 2, 2, 64, 48, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()

    def run():
        out, state = forward(x, offsets, initial, final_state=True)
        grads = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
        torch.cuda.synchronize()
        return out, state, grads
    good = run()
    x[what][(at, 1) if what in ("g", "beta") else (at, 1, 5)] = float(value)
    bad = run()
    keep = torch.ones(x["v"].shape[0], dtype=torch.bool, device="cuda")
    keep[200:270] = False
    for a, b in zip((good[0], *good[2][:5]), (bad[0], *bad[2][:5])):
        assert torch.equal(a[keep], b[keep]) and torch.equal(a[:, 0], b[:, 0])
    for a, b in ((good[1], bad[1]), (good[2][5], bad[2][5])):
        assert torch.equal(a[[0, 2, 3]], b[[0, 2, 3]]) and torch.equal(a[1, 0], b[1, 0])
    chunk = 32 if dtype == FP32 else 64
    assert torch.equal(good[0][200: 200 + 69 // chunk * chunk], bad[0][200: 200 + 69 // chunk * chunk])
    assert not torch.isfinite(bad[0][at, 1]).all() or (what in ("k", "g", "beta") and not torch.isfinite(bad[1][1, 1]).all())


def test_empty_calls(gpu):
    x, offsets, initial = inputs(11, [0, 0], 1, 2, 32, 24, BF16)
    out, state = forward(x, offsets, initial, final_state=True)
    assert out.shape == (0, 2, 24) and torch.equal(state, initial)
    got = dws.delta_rule_backward(torch.empty_like(x["v"]), *(x[a] for a in NAMES), offsets=offsets, initial_state=initial,
                                  d_final_state=initial)
    assert torch.equal(got[5], initial.to(BF16)) and got[0].numel() == 0
    pool = initial.clone()
    dws.delta_rule_step(*(x[a] for a in NAMES), pool)
    assert torch.equal(pool, initial)


def test_offsets_that_decrease_touch_nothing_outside(gpu):
    """Wrong offsets give unspecified values, inside the arrays."""
    x, _, initial = inputs(12, [200], 1, 2, 32, 24, BF16, init=False)
    for bad in ([0, 300, 100, 200], [-50, 20, 10, 1 << 40], [200, 0, 200, 0]):
        offsets = torch.tensor(bad, dtype=torch.int64, device="cuda")
        guard = torch.full((600, 2, 24), 5.0, dtype=BF16, device="cuda")
        out, state = forward(x, offsets, None, out=guard[200:400], final_state=True)
        assert state.shape[0] == 3 and (guard[:200] == 5).all() and (guard[400:] == 5).all()
        dws.delta_rule_backward(out.contiguous(), *(x[a] for a in NAMES), offsets=offsets)
        torch.cuda.synchronize()


# sequences, tokens of each, heads_qk, value heads a key head, dim_k, dim_v; the last ones have more heads than the
# device has compute units
STEPS = [(1, 1, 1, 1, 1, 1), (3, 1, 2, 4, 64, 64), (5, 2, 1, 3, 128, 128), (2, 7, 1, 1, 256, 255), (4, 3, 2, 2, 40, 100),
         (130, 1, 1, 2, 64, 64), (43, 2, 2, 3, 72, 36), (150, 1, 2, 1, 128, 128), (70, 3, 4, 1, 256, 132), (300, 1, 1, 1, 24, 31)]


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("n,tokens,hk,hv,dk,dv", [(n, t, hk, hk * r, dk, dv) for n, t, hk, r, dk, dv in STEPS])
def test_step(gpu, n, tokens, hk, hv, dk, dv, dtype):
    note(f"delta step {n} {tokens} {hk} {hv} {dk} {dv} {dtype}")
    x, offsets, initial = inputs(13, [tokens] * n, hk, hv, dk, dv, dtype)
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), initial.double().cpu(), dk ** -0.5)
    pool = torch.full((n + 3, hv, dk, dv), 9.0, device="cuda")
    slots = torch.randperm(n + 3, generator=torch.Generator().manual_seed(1))[:n].to(torch.int32).cuda()
    pool[slots.long()] = initial
    out = dws.delta_rule_step(*(x[a] for a in NAMES), pool, slots=slots)
    close(out, want, dtype, "out")
    close(pool[slots.long()], final, FP32, "state")
    rest = torch.ones(n + 3, dtype=torch.bool)
    rest[slots.long().cpu()] = False
    assert (pool[rest.cuda()] == 9).all()
    again = initial.clone()
    assert torch.equal(dws.delta_rule_step(*(x[a] for a in NAMES), again), out)
    assert torch.equal(again, pool[slots.long()])


@pytest.mark.parametrize("dv", [64, 128])
def test_step_of_a_large_batch(gpu, dv):
    """States of more than 128 MB, which are read and written past the caches."""
    n, hv, dk = 1100 * 64 // dv, 2, 256
    assert n * hv * dk * dv * 4 >= 128 << 20
    x, offsets, _ = inputs(22, [2] * n, 1, hv, dk, dv, BF16, init=False)
    gen = torch.Generator(device="cuda").manual_seed(5)
    pool = 0.3 * torch.randn(n + 1, hv, dk, dv, device="cuda", generator=gen)
    first = pool.clone()
    slots = torch.arange(n, 0, -1, dtype=torch.int32, device="cuda")
    out = dws.delta_rule_step(*(x[a] for a in NAMES), pool, slots=slots)
    assert torch.equal(pool[0], first[0])
    for i in (0, 1, n // 2, n - 1):
        y = {a: x[a][2 * i: 2 * i + 2] for a in NAMES}
        want, final = reference(*(y[a] for a in NAMES), [0, 2], first[n - i: n - i + 1].double().cpu(), 1 / 16)
        close(out[2 * i: 2 * i + 2], want, BF16, "out")
        close(pool[n - i: n - i + 1], final, FP32, "state")


@pytest.mark.parametrize("whole", [False, True])
def test_slots_that_leave_sequences_out(gpu, whole):
    """A slot below 0, outside the pool or named before: the sequence's rows and the states stay as they were."""
    lens = [3, 2, 4, 1, 3, 2]
    x, offsets, _ = inputs(14, lens, 1, 2, 32, 16, FP32)
    slots = torch.tensor([4, -1, 2, 4, 7, 0], dtype=torch.int32, device="cuda")
    pool = 0.3 * torch.randn(7, 2, 32, 16, device="cuda")
    before = pool.clone()
    out = torch.full(x["v"].shape, 3.0, device="cuda")
    if whole:
        dws.delta_rule(*(x[a] for a in NAMES), offsets=offsets, initial_state=pool, final_state=pool, slots=slots, out=out)
    else:
        dws.delta_rule_step(*(x[a] for a in NAMES), pool, slots=slots, offsets=offsets, out=out)
    first = torch.zeros(6, 2, 32, 16, dtype=torch.float64)
    taken = {0: 4, 2: 2, 5: 0}
    for i, s in taken.items():
        first[i] = before[s].double().cpu()
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), first, 32 ** -0.5)
    ends = offsets.tolist()
    for i in range(6):
        rows = slice(ends[i], ends[i + 1])
        if i in taken:
            close(out[rows], want[rows], FP32, "out")
            close(pool[taken[i]], final[i], FP32, "state")
        else:
            assert (out[rows] == 3).all()
    for s in (1, 3, 5, 6):
        assert torch.equal(pool[s], before[s])


@pytest.mark.parametrize("n,most,hk,hv,dk,dv,dtype", [(50000, 4, 1, 2, 16, 16, BF16), (3000, 70, 2, 2, 96, 40, FP16),
                                                      (1, 120000, 1, 1, 64, 64, BF16), (300, 200, 2, 4, 136, 64, FP32)])
def test_chunks_and_steps_agree(gpu, n, most, hk, hv, dk, dv, dtype):
    """The two forms against each other at sizes that the definition takes too long for: very many and very long
    sequences. (As tolerance the one of two results of the type, each off by its own.)"""
    note(f"delta chunks and steps {n} {most} {dtype}")
    gen = torch.Generator().manual_seed(25)
    lens = torch.randint(0, most + 1, (n,), generator=gen).tolist() if n > 1 else [most]
    x, offsets, initial = inputs(26, lens, hk, hv, dk, dv, dtype)
    out, final = forward(x, offsets, initial, final_state=True)
    pool = initial.clone()
    stepped = dws.delta_rule_step(*(x[a] for a in NAMES), pool, offsets=offsets)
    torch.cuda.synchronize()
    close(out, stepped, dtype, "dg")
    close(forward(x, offsets, initial), stepped, dtype, "dg")
    # both are off by the fp32 tolerance
    off = (final - pool).double().norm() / pool.double().norm()
    assert off <= 2 * tolerance(dtype, "state"), off


def test_prefill_then_steps(gpu):
    """A prompt in two calls and tokens one by one, states in a pool, are the sequence in one."""
    lens = [150, 97]
    x, offsets, _ = inputs(15, lens, 2, 4, 64, 48, BF16, init=False)
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), None, 64 ** -0.5)
    pool = torch.randn(5, 4, 64, 48, device="cuda")
    slots = torch.tensor([3, 1], dtype=torch.int32, device="cuda")
    cuts = [(0, 70), (70, 90)]
    outs = [[], []]

    def part(a, b):
        rows = torch.cat([torch.arange(s + a, s + b) for s in (0, 150)]).cuda()
        return {y: x[y][rows] for y in NAMES}, torch.tensor([0, b - a, 2 * (b - a)], device="cuda")

    for i, (a, b) in enumerate(cuts):
        y, off = part(a, b)
        o, _ = dws.delta_rule(*(y[z] for z in NAMES), offsets=off, initial_state=pool if i else None, final_state=pool,
                              slots=slots)
        for s in range(2):
            outs[s].append(o[s * (b - a):(s + 1) * (b - a)])
    for t in range(90, 97):
        y, off = part(t, t + 1)
        o = dws.delta_rule_step(*(y[z] for z in NAMES), pool, slots=slots)
        for s in range(2):
            outs[s].append(o[s: s + 1])
    for s, start in enumerate((0, 150)):
        close(torch.cat(outs[s]), want[start: start + 97], BF16, "out")
    _, final = reference(*(x[a] for a in NAMES), [0, 97], None, 64 ** -0.5)
    close(pool[3], final[0], BF16, "state")


def test_far_states(gpu):
    """States whose place in the pool is beyond 2^32 bytes and 2^31 elements."""
    hv, dk, dv = 1, 256, 256
    count = (1 << 31) // (dk * dv) + 5
    pool = torch.empty(count, hv, dk, dv, device="cuda")
    x, offsets, initial = inputs(16, [3, 2], 1, hv, dk, dv, FP32)
    slots = torch.tensor([count - 1, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = initial
    want, final = reference(*(x[a] for a in NAMES), offsets.tolist(), initial.double().cpu(), 1 / 16)
    close(dws.delta_rule_step(*(x[a] for a in NAMES), pool, slots=slots, offsets=offsets), want, FP32, "out")
    close(pool[slots.long()], final, FP32, "state")
    pool[slots.long()] = initial
    out, _ = dws.delta_rule(*(x[a] for a in NAMES), offsets=offsets, initial_state=pool, final_state=pool, slots=slots)
    close(out, want, FP32, "out")
    close(pool[slots.long()], final, FP32, "state")


def test_repeats_bit_for_bit(gpu):
    x, offsets, initial = inputs(17, [500, 129], 2, 6, 64, 64, BF16)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    first = None
    for _ in range(4):
        got = forward(x, offsets, initial, final_state=True)
        got += dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(got, first))


def test_graphs_and_streams(gpu):
    """Each call captured once and replayed between eager calls and on its own beside them; two graphs and a stream at
    once do not share memory."""
    x, offsets, initial = inputs(18, [200, 65], 2, 4, 64, 64, BF16)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(2)).to(BF16).cuda()
    args = [x[a] for a in NAMES]

    def everything(pool):
        out, final = dws.delta_rule(*args, offsets=offsets, initial_state=initial, final_state=True)
        grads = dws.delta_rule_backward(d_out, *args, offsets=offsets, initial_state=initial)
        stepped = dws.delta_rule_step(*(y[:2] for y in args), pool)
        return [out, final, *grads, stepped, pool]

    want = [t.clone() for t in everything(initial.clone())]
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        pool = initial.clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = everything(pool)
        graphs.append((graph, got, pool))
    side = torch.cuda.Stream()
    for _ in range(3):
        for _, got, pool in graphs:
            for t in got:
                t.zero_()
            pool.copy_(initial)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            aside = everything(initial.clone())
        for graph, _, _ in graphs:
            graph.replay()
        eager = everything(initial.clone())
        torch.cuda.synchronize()
        for got in (aside, eager, graphs[0][1], graphs[1][1]):
            assert all(torch.equal(a, b) for a, b in zip(got, want))
    # another stream by its handle: what the binding allocates belongs to that stream
    for _ in range(3):
        out, final = dws.delta_rule(*args, offsets=offsets, initial_state=initial, final_state=True,
                                    stream=side.cuda_stream)
        junk = [torch.full_like(out, 3.0) for _ in range(4)]
        side.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(final, want[1]) and len(junk) == 4


@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("dtype,dk,dv", [(FP32, 65, 24), (FP32, 100, 36), (FP32, 12, 4), (FP32, 36, 17), (FP32, 130, 100),
                                         (BF16, 12, 20), (BF16, 100, 65), (FP16, 65, 36)])
def test_heads_do_not_meet_at_their_rows_ends(gpu, what, dtype, dk, dv):
    """Rows that end inside a fragment: the next head's first elements, infinite here, change no bit of the head before."""
    x, offsets, initial = inputs(31, [70, 40], 2, 2, dk, dv, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()

    def run():
        out, state = forward(x, offsets, initial, final_state=True)
        return [out, state, *dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)]
    good = run()
    x[what][50, 1, :4] = float("inf")
    for a, b in zip(good, run()):
        assert torch.equal(a[:, 0], b[:, 0])


@pytest.mark.parametrize("dtype,dk,dv", [(FP32, 100, 36), (FP32, 36, 100), (FP32, 65, 17), (BF16, 40, 104), (FP16, 100, 36)])
def test_what_lies_between_strided_rows_is_not_used(gpu, dtype, dk, dv):
    """Parts of buffers that hold NaN everywhere else give the bits of the arrays alone."""
    x, offsets, initial = inputs(32, [70, 33], 2, 4, dk, dv, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()

    def run(y, d):
        out, state = forward(y, offsets, initial, final_state=True)
        return [out, state, *dws.delta_rule_backward(d, *(y[a] for a in NAMES), offsets=offsets, initial_state=initial)]

    def inside(t, gap):
        n, heads, dim = t.shape
        part = torch.full((n + 2, heads + 1, dim + gap), float("nan"), dtype=t.dtype, device="cuda")[1: n + 1, :heads, :dim]
        return part.copy_(t)
    want = run(x, d_out)
    for gap in (16, 12, 1):          # with 16-byte units kept, kept for fp32 only, and not
        y = dict(x, **{a: inside(x[a], gap) for a in ("q", "k", "v")})
        for a, b in zip(run(y, inside(d_out, gap)), want):
            assert torch.equal(a, b)


CODES = {FP32: dws.FLOAT32, FP16: dws.FLOAT16, BF16: dws.BFLOAT16}


def rows_of(t):
    return dws.Rows(t.data_ptr(), t.stride(0), t.stride(1))


def c_arguments(x, n_seqs, **more):
    """dws_delta_rule_args, for what the binding does not pass."""
    a = dws.DeltaRuleArgs()
    a.tokens, a.heads_qk, a.dim_k = x["q"].shape
    a.n_seqs, a.heads_v, a.dim_v = n_seqs, x["v"].shape[1], x["v"].shape[2]
    a.dtype, a.g_dtype, a.beta_dtype = (CODES[x[b].dtype] for b in ("q", "g", "beta"))
    a.scale = a.dim_k ** -0.5
    for name, value in {**{b: rows_of(x[b]) for b in NAMES}, **more}.items():
        setattr(a, name, value)
    return a


def c_call(name, a, backward=None):
    """The call by its name, with a workspace of its own where one is needed (`backward` 0 or 1)."""
    lib = dws.load_library()
    if backward is not None:
        need = ctypes.c_size_t(0)
        assert lib.dws_delta_rule_workspace(ctypes.byref(a), backward, ctypes.byref(need)) == dws.OK
        work = torch.empty(need.value, dtype=torch.uint8, device="cuda")
        a.d_workspace, a.workspace_bytes = work.data_ptr(), need.value
    status = getattr(lib, name)(ctypes.byref(a), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    return status


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("head,lens,tail", [(0, [2, 1], 0), (3, [2, 1], 0), (0, [2, 1], 1), (70, [1, 0, 4], 1500), (5, [0], 2)])
def test_step_clears_the_rows_in_no_sequence(gpu, dtype, head, lens, tail):
    """zero_rest: those before the first sequence and behind the last, and no others; without it they stay."""
    x, offsets, initial = inputs(33, lens, 1, 2, 32, 23, dtype, tail=head + tail)
    offsets += head
    end = head + sum(lens)
    for a in NAMES:
        x[a][:head] = x[a][end:] = float("nan")
    pool = initial.clone()
    want = dws.delta_rule_step(*(x[a] for a in NAMES), pool, offsets=offsets)
    for rest in (1, 0):
        state = initial.clone()
        wide = torch.full((x["v"].shape[0] + 2, 3, 23), 5.0, dtype=dtype, device="cuda")
        out = wide[1:-1, :2]
        a = c_arguments(x, len(lens), out=rows_of(out), d_offsets=offsets.data_ptr(), d_initial_state=state.data_ptr(),
                        d_final_state=state.data_ptr(), zero_rest=rest)
        assert c_call("dws_delta_rule_step", a) == dws.OK
        assert torch.equal(out[head:end], want[head:end]) and torch.equal(state, pool)
        left = 0 if rest else 5
        assert (out[:head] == left).all() and (out[end:] == left).all()
        assert (wide[:, 2] == 5).all() and (wide[0] == 5).all() and (wide[-1] == 5).all()


def test_in_an_autograd_function(gpu):
    """The calls as a model's training step makes them, on tensors that require gradients: refused outside, and inside a
    function's forward and backward the gradients of the definition."""
    x, offsets, initial = inputs(34, [40, 25], 1, 2, 32, 16, FP32)

    class Rule(torch.autograd.Function):
        @staticmethod
        def forward(ctx, *args):
            ctx.save_for_backward(*args)
            return dws.delta_rule(*args[:5], offsets=offsets, initial_state=args[5], final_state=True)

        @staticmethod
        def backward(ctx, d_out, d_final):
            *args, s = ctx.saved_tensors
            return dws.delta_rule_backward(d_out, *args, offsets=offsets, initial_state=s, d_final_state=d_final)

    leaves = [x[a].requires_grad_() for a in NAMES] + [initial.requires_grad_()]
    with pytest.raises(RuntimeError, match="no graph"):
        dws.delta_rule(*leaves[:5], offsets=offsets)
    with pytest.raises(RuntimeError, match="no graph"):
        dws.delta_rule_step(*leaves[:5], initial.detach(), offsets=offsets)
    out, state = Rule.apply(*leaves)
    gen = torch.Generator().manual_seed(3)
    d_out = torch.randn(out.shape, generator=gen).cuda()
    d_final = torch.randn(state.shape, generator=gen).cuda()
    got = torch.autograd.grad((out * d_out).sum() + (state * d_final).sum(), leaves)
    want = gradients({a: x[a].detach() for a in NAMES}, offsets, initial.detach(), 32 ** -0.5, d_out, d_final)
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
        close(a, b, FP32, what)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([70, 0, 33], 1, 2, 64, 40), ([129], 2, 2, 128, 128), ([65, 1], 1, 3, 136, 17)])
def test_gradients_of_fp32_gates_and_states(gpu, lens, hk, hv, dk, dv, dtype):
    """fp32_grads: the same values before their rounding, nearer to the definition; rows in no sequence 0 as well."""
    x, offsets, initial = inputs(35, lens, hk, hv, dk, dv, dtype, tail=75)
    offsets += 5
    gen = torch.Generator().manual_seed(3)
    d_out = torch.randn(x["v"].shape, generator=gen).to(dtype).cuda()
    d_final = 0.3 * torch.randn(initial.shape, generator=gen).cuda()
    args = (d_out, *(x[a] for a in NAMES))
    more = {"offsets": offsets, "initial_state": initial, "d_final_state": d_final}
    narrow = dws.delta_rule_backward(*args, **more)
    dirty = [torch.full_like(x["g"], float("nan")) for _ in range(4)]      # what new tensors find in their memory
    del dirty
    wide = dws.delta_rule_backward(*args, **more, fp32_grads=True)
    want = gradients(x, offsets, initial, dk ** -0.5, d_out, d_final)
    for what, a, b, c in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), narrow, wide, want):
        assert b.dtype == (dtype if what in ("dq", "dk", "dv") else FP32) and a.dtype == dtype
        assert torch.equal(b.to(dtype), a), what
        close(b, c, dtype, what)
        if dtype != FP32 and b.dtype == FP32:
            assert (b.double().cpu() - c).norm() < (a.double().cpu() - c).norm(), what
        if what != "d_initial":
            assert (b[:5] == 0).all() and (b[5 + sum(lens):] == 0).all(), what


@pytest.mark.parametrize("dtype", [BF16, FP16])
def test_segments_pass_the_states_gradient_on(gpu, dtype):
    """A sequence differentiated in three parts, each with the state's gradient of the one behind it, is the sequence in one."""
    cuts = [0, 128, 320, 365]
    x, offsets, initial = inputs(36, [cuts[-1]], 1, 2, 64, 48, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    states = [initial]
    parts = [{a: x[a][b:e] for a in NAMES} for b, e in zip(cuts, cuts[1:])]
    for y in parts:
        states.append(dws.delta_rule(*(y[a] for a in NAMES), initial_state=states[-1], final_state=True)[1])
    with pytest.raises(ValueError):
        dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), initial_state=initial, d_final_state=initial.to(dtype))
    got, ds = [], None
    for i in (2, 1, 0):
        *grads, ds = dws.delta_rule_backward(d_out[cuts[i]: cuts[i + 1]], *(parts[i][a] for a in NAMES),
                                             initial_state=states[i], d_final_state=ds, fp32_grads=True)
        got.insert(0, grads)
    want = gradients(x, offsets, initial, 64 ** -0.5, d_out, None)
    for i, what in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        close(torch.cat([g[i] for g in got]), want[i], dtype, what)
    close(ds, want[5], dtype, "d_initial")


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("n,hk,hv,dk,dv", [(64, 2, 4, 64, 64), (41, 1, 2, 128, 96), (32, 1, 2, 200, 64)])
def test_the_states_gradient_of_one_chunk(gpu, n, hk, hv, dk, dv, dtype):
    """Nothing on its way is rounded to one 16-bit part: P, the inverse, dU and the two operands of the last products are
    in two, each off by 2^-16 (fp16 2^-22), and the sums are fp32's, as tolerance() counts them.

    An fp16 part below 2^-14 is off by up to 2^-25, however small it is, which the second parts of small operands are.
    With all factors e^G and beta at most 1, and norms ||.|| of the matrices, the result is Q^T e - K^T y, with
    y = T^T dU and dU = P^T dO scaled: e and y off by 2^-25 an element add 2^-25 sqrt(n dv) (||Q|| + ||K||), dU's
    2^-25 sqrt(n dv) go through T and K, T's 2^-25 n (an n x n matrix) meet dU and K, and P's meet dO, T and K."""
    x, offsets, initial = inputs(37, [n], hk, hv, dk, dv, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), initial_state=initial, fp32_grads=True)[5].double().cpu()
    want = gradients(x, offsets, initial, dk ** -0.5, d_out, None)[5]
    tiny = 0.0
    if dtype == FP16:
        y = {a: x[a].double().cpu() for a in NAMES}
        norm = torch.linalg.matrix_norm
        for h in range(hv):
            q, k, d_o = y["q"][:, h * hk // hv], y["k"][:, h * hk // hv], d_out[:, h].double().cpu()
            total = y["g"][:, h].cumsum(0)
            decay = (total[:, None] - total[None, :]).tril().exp().tril()
            t = torch.linalg.inv(torch.eye(n) + (y["beta"][:, h, None] * decay * (k @ k.T)).tril(-1))
            d_u = dk ** -0.5 * (decay * (q @ k.T)).T @ d_o
            nq, nk, nt, nu, no = (norm(z, 2).item() for z in (q, k, t, d_u, d_o))
            tiny += (2.0 ** -25 * ((n * dv) ** 0.5 * (nq + nk * (1 + nt)) + n * nk * (nu + nt * no))) ** 2
    off, most = (got - want).norm().item(), 5 * (2.0 ** -16 if dtype == BF16 else 2.0 ** -22) + tolerance(FP32, "state")
    print(f"off by {off / want.norm():.3g}, {most + tiny ** 0.5 / want.norm().item():.3g} allowed")
    assert off <= most * want.norm().item() + tiny ** 0.5


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([130, 1, 0, 64], 1, 2, 64, 48), ([200], 2, 2, 128, 128), ([70], 1, 1, 200, 40),
                                              ([40] * 40, 4, 8, 96, 64)])
def test_precise_outputs(gpu, lens, hk, hv, dk, dv, dtype):
    """The same bits whether the final state is asked for or not."""
    x, offsets, initial = inputs(38, lens, hk, hv, dk, dv, dtype, tail=3)
    want, _ = forward(x, offsets, initial, final_state=True)
    assert torch.equal(forward(x, offsets, initial, precise=True), want)
    assert torch.equal(forward(x, offsets, initial, precise=True, final_state=True)[0], want)
    if dtype == FP32:
        assert torch.equal(forward(x, offsets, initial), want)


@pytest.mark.parametrize("n,each,hk,hv,dk,dv,dtype", [(3, 50, 1, 2, 40, 24, FP32), (70, 33, 1, 2, 64, 32, BF16),
                                                      (200, 1, 2, 2, 32, 40, FP16), (5, 129, 2, 4, 136, 17, BF16),
                                                      (4, 0, 1, 1, 16, 16, BF16), (300, 65, 1, 1, 64, 64, BF16)])
def test_equal_shares_without_offsets(gpu, n, each, hk, hv, dk, dv, dtype):
    """No offsets: tokens / n_seqs rows a sequence, with the bits of the offsets that say so."""
    note(f"delta equal shares {n} {each} {dtype}")
    x, offsets, initial = inputs(39, [each] * n, hk, hv, dk, dv, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(6)).to(dtype).cuda()
    d_final = 0.3 * torch.randn(initial.shape, generator=torch.Generator().manual_seed(7)).cuda()
    pool = initial.clone()
    more = {"offsets": offsets, "initial_state": initial}
    want = [*forward(x, offsets, initial, final_state=True), dws.delta_rule_step(*(x[a] for a in NAMES), pool, offsets=offsets),
            pool, *dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), **more, d_final_state=d_final)]
    out, final, stepped, state, *grads = [torch.full_like(t, 3.0) for t in want]
    state.copy_(initial)
    names = ("q_grad", "k_grad", "v_grad", "g_grad", "beta_grad")
    for rest in (0, 1):
        a = c_arguments(x, n, out=rows_of(out), d_initial_state=initial.data_ptr(), d_final_state=final.data_ptr(), zero_rest=rest,
                        out_grad=rows_of(d_out), d_final_grad=d_final.data_ptr(), d_initial_grad=grads[5].data_ptr(),
                        **{name: rows_of(t) for name, t in zip(names, grads)})
        assert c_call("dws_delta_rule", a, 0) == dws.OK
        assert c_call("dws_delta_rule_backward", a, 1) == dws.OK
    a.out, a.d_initial_state, a.d_final_state = rows_of(stepped), state.data_ptr(), state.data_ptr()
    assert c_call("dws_delta_rule_step", a) == dws.OK
    for got, t in zip((out, final, stepped, state, *grads), want):
        assert torch.equal(got, t)


@pytest.mark.parametrize("whole", [False, True])
def test_many_slots(gpu, whole):
    """Tens of thousands of sequences on a pool: duplicates and places outside it among them, each found by a search of
    the slots before its own."""
    n, count, dk, dv = 40000, 30000, 16, 16
    lens = [1] * n
    x, offsets, _ = inputs(40, lens, 1, 1, dk, dv, BF16, init=False)
    gen = torch.Generator().manual_seed(2)
    slots = torch.randint(-5, count + 5, (n,), generator=gen).to(torch.int32)
    pool = 0.3 * torch.randn(count, 1, dk, dv, generator=gen)
    seen, first = {}, []
    for i, s in enumerate(slots.tolist()):
        first.append(0 <= s < count and s not in seen)
        seen.setdefault(s, i)
    first = torch.tensor(first)
    assert 10000 < int(first.sum()) < 30000
    out = torch.full(x["v"].shape, 3.0, dtype=BF16, device="cuda")
    state, where = pool.cuda(), slots.cuda()
    args = [x[a] for a in NAMES]
    if whole:
        dws.delta_rule(*args, offsets=offsets, initial_state=state, final_state=state, slots=where, out=out)
    else:
        dws.delta_rule_step(*args, state, slots=where, out=out)
    assert (out[~first.cuda()] == 3).all()
    # the sequences that take part, with states of their own and no slots
    some = first.nonzero().reshape(-1)
    alone = pool[slots[some].long()].cuda()
    some_args = [t[some.cuda()] for t in args]
    if whole:
        want, final = dws.delta_rule(*some_args, offsets=torch.arange(len(some) + 1, device="cuda"), initial_state=alone,
                                     final_state=True)
    else:
        want, final = dws.delta_rule_step(*some_args, alone), alone
    assert torch.equal(out[first.cuda()], want)
    wanted = pool.clone()
    wanted[slots[some].long()] = final.cpu()
    assert torch.equal(state.cpu(), wanted)


def test_gradients_with_a_workspace_beyond_32_bits(gpu):
    """A long sequence before a short one: the short one's gradients are those it has alone, and the long one's last part
    has those it has as a sequence of its own behind the state before it."""
    long, last, short, hk, hv, dk = 100032, 960, 70, 2, 16, 128
    gen = torch.Generator(device="cuda").manual_seed(41)
    n = long + short

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    x = {a: torch.nn.functional.normalize(normal(n, hk, dk), dim=-1).to(BF16) for a in ("q", "k")}
    x["v"], d_out = normal(n, hv, dk).to(BF16), normal(n, hv, dk).to(BF16)
    x["g"], x["beta"] = -0.1 * torch.rand(n, hv, generator=gen, device="cuda"), torch.rand(n, hv, generator=gen, device="cuda").to(BF16)
    offsets = torch.tensor([0, long, n], device="cuda")
    a = c_arguments(x, 2, d_offsets=offsets.data_ptr())
    need = ctypes.c_size_t(0)
    assert dws.load_library().dws_delta_rule_workspace(ctypes.byref(a), 1, ctypes.byref(need)) == dws.OK
    assert need.value > 1 << 32
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets)[:5]
    out = forward(x, offsets, None)

    def part(rows):
        return {a: x[a][rows] for a in NAMES}
    rows = slice(long, n)
    alone = dws.delta_rule_backward(d_out[rows], *part(rows).values())[:5]
    assert torch.equal(out[rows], forward(part(rows), None, None))
    for a, b in zip(got, alone):
        assert torch.equal(a[rows], b)
    before, rows = slice(0, long - last), slice(long - last, long)
    state = dws.delta_rule(*part(before).values(), final_state=True)[1]
    close(out[rows], forward(part(rows), None, state), BF16, "dg")
    alone = dws.delta_rule_backward(d_out[rows], *part(rows).values(), initial_state=state)[:5]
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta"), got, alone):
        off = ((a[rows].double() - b.double()).norm() / b.double().norm()).item()
        assert off <= 2 * tolerance(BF16, what), (what, off)          # both are off by the tolerance


def test_rows_far_apart(gpu):
    """Tokens whose rows are beyond 2^31 elements and 2^32 bytes of their first."""
    n, hk, hv, dk, dv, stride = 1100, 1, 2, 64, 32, 1 << 21
    x, offsets, initial = inputs(42, [700, n - 700], hk, hv, dk, dv, BF16)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).to(BF16).cuda()
    far = torch.empty(n * stride, dtype=BF16, device="cuda")
    y, at = dict(x), 0
    for a in ("q", "k", "v"):
        heads, dim = x[a].shape[1:]
        y[a] = far.as_strided((n, heads, dim), (stride, dim, 1), at)
        y[a].copy_(x[a])
        at += heads * dim
    d_far = far.as_strided((n, hv, dv), (stride, dv, 1), at)
    d_far.copy_(d_out)
    want, final = forward(x, offsets, initial, final_state=True)
    got, state = forward(y, offsets, initial, final_state=True)
    assert torch.equal(got, want) and torch.equal(state, final)
    for a, b in zip(dws.delta_rule_backward(d_far, *(y[a] for a in NAMES), offsets=offsets, initial_state=initial),
                    dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial)):
        assert torch.equal(a, b)
    pool, far_pool = initial.clone(), initial.clone()
    assert torch.equal(dws.delta_rule_step(*(y[a] for a in NAMES), far_pool, offsets=offsets),
                       dws.delta_rule_step(*(x[a] for a in NAMES), pool, offsets=offsets))
    assert torch.equal(pool, far_pool)
    # and a far output, in an array of its own
    wide = torch.empty(n * stride, dtype=BF16, device="cuda").as_strided((n, hv, dv), (stride, dv, 1), 8)
    forward(x, offsets, initial, out=wide, final_state=True)
    assert torch.equal(wide, want)


@pytest.mark.parametrize("dtype", [FP32, BF16, FP16])
@pytest.mark.parametrize("lens,hk,hv,dk,dv", [([70, 0, 33], 1, 2, 64, 40), ([301], 2, 2, 128, 128), ([200, 65], 1, 2, 96, 64),
                                              ([90], 1, 1, 200, 64), ([20, 45] * 20, 4, 8, 128, 64)])
def test_precise_gradients(gpu, lens, hk, hv, dk, dv, dtype):
    """No operand in one part: a rounded gradient is its rounding away from the definition, and one in fp32 at most six
    two-part products deep (P, the inverse, dU, Z, S, dS'), off by 2^-16 each and double where sums cancel. (fp16's
    second parts are below 2^-14, where they lose digits, but not more than bf16's have.)"""
    x, offsets, initial = inputs(43, lens, hk, hv, dk, dv, dtype)
    d_out = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    got = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial, fp32_grads=True, precise=True)
    want = gradients(x, offsets, initial, dk ** -0.5, d_out, None)
    fine = 12 * 2.0 ** -16 if dtype != FP32 else 0.0
    for what, a, b in zip(("dq", "dk", "dv", "dg", "dbeta", "d_initial"), got, want):
        close(a, b, dtype, what)
        off, rounding = (a.double().cpu() - b).norm().item(), (b.to(a.dtype).double() - b).norm().item()
        most = rounding + (fine + tolerance(FP32, "state")) * b.norm().item()
        assert off <= most, f"{what}: off by {off / rounding:.3f} times its rounding, {off / b.norm().item():.3g} of its norm"
    if dk > 128 or dtype == FP32:        # as without
        plain = dws.delta_rule_backward(d_out, *(x[a] for a in NAMES), offsets=offsets, initial_state=initial, fp32_grads=True)
        assert all(torch.equal(a, b) for a, b in zip(got, plain))
