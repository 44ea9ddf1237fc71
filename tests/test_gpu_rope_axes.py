"""GPU: the multi-axis rotation (RopeAxes.apply, rope_axes) against its 64-bit definition, element by element, and its
gradients against the formula's, differences and autograd's own bookkeeping."""
import pytest
import torch

import serving_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def aa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import packed_sequence_rope_gb300 as pkg
    return pkg


def _data(T, Hq, Hk, D, axes, seed=1, far=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(-far if far else 0, far if far else 5000, (axes, T), generator=g, dtype=torch.int64)
    return r(T, Hq, D), r(T, Hk, D), pos.to(torch.int32).cuda()


def _check(y, x, pos, rope, theta, half, inverse=False):
    want = ref.turn(x, pos, rope.axis_of_pair, theta, half, inverse)
    err = (y.double().cpu() - want).abs() - ref.turn_bound(want, x, half)
    assert err.max() <= 0, f"beyond the bound by {err.max():.3e}"


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 63, 257, 1400])
@pytest.mark.parametrize("D,sections,inter", [(128, (16, 24, 24), False), (64, (8, 12, 12), True), (128, (64,), False),
                                              (64, (0, 32), False), (128, (1, 2, 3, 58), True)])
@pytest.mark.parametrize("half", [False, True])
def test_matches_definition(aa, T, D, sections, inter, half):
    layout = aa.ROPE_HALF if half else aa.ROPE_ADJACENT
    rope = aa.RopeAxes(D, sections, base=5e5, layout=layout, interleaved=inter)
    theta = [5e5 ** (-2.0 * p / D) for p in range(D // 2)]
    for Hq, Hk in ((4, 1), (5, 3), (32, 8)):
        q, k, pos = _data(T, Hq, Hk, D, rope.num_axes)
        yq, yk = rope.apply(pos, q, k)
        _check(yq, q, pos, rope, theta, half)
        _check(yk, k, pos, rope, theta, half)
        _check(rope.apply(pos, yq, inverse=True), yq, pos, rope, theta, half, inverse=True)


def test_far_and_negative_positions(aa):
    rope = aa.RopeAxes(128, (32, 32), base=1e4)
    theta = [1e4 ** (-2.0 * p / 128) for p in range(64)]
    q, k, pos = _data(300, 2, 1, 128, 2, far=2 ** 30)
    yq, yk = rope.apply(pos, q, k)
    _check(yq, q, pos, rope, theta, False)
    _check(yk, k, pos, rope, theta, False)


def test_given_frequencies_and_zero_ones(aa):
    theta = [0.0 if p % 3 == 0 else 0.9 ** p for p in range(32)]
    rope = aa.RopeAxes(64, (32,), theta=theta, layout=aa.ROPE_HALF)
    q, k, pos = _data(33, 3, 2, 64, 1)
    yq, _ = rope.apply(pos[0], q, k)  # [T] for a single axis
    _check(yq, q, pos, rope, theta, True)
    still = [p for p in range(32) if theta[p] == 0.0]
    assert torch.equal(yq[..., still], q[..., still])


def test_agrees_with_a_plan_on_one_axis(aa):
    # the same rotation as aa_rope_apply for the plan's positions, up to each one's rounding
    T, D = 700, 128
    q, _, _ = _data(T, 4, 1, D, 1)
    with aa.Plan([1, 300, 700], T, 4, 4, D, 5e6) as plan:
        want = plan.rope_apply(q)
        pos = torch.from_numpy(plan.metadata()[1]).cuda()
    got = aa.RopeAxes(D, (64,), base=5e6).apply(pos, q)
    assert ((got.double() - want.double()).abs() <= want.double().abs() * 2.0 ** -7 + 4e-4).all()


def test_slices_in_place_and_odd_strides(aa):
    T, Hq, Hk, D = 77, 6, 2, 128
    rope = aa.RopeAxes(D, (16, 24, 24), base=1e4, layout=aa.ROPE_HALF)
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(T, Hq + 2 * Hk, D, generator=g).to(torch.bfloat16).cuda()
    _, _, pos = _data(T, 1, 1, D, 3)
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    before = qkv.clone()
    yq, yk = rope.apply(pos, q, k)
    assert torch.equal(qkv, before)
    qc, kc = q.contiguous(), k.contiguous()
    wq, wk = rope.apply(pos, qc, kc)
    assert torch.equal(yq, wq) and torch.equal(yk, wk)
    # in place
    rope.apply(pos, qc, kc, out_q=qc, out_k=kc)
    assert torch.equal(qc, wq) and torch.equal(kc, wk)
    # a transposed, an unaligned and a broadcast input
    t = q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    assert torch.equal(rope.apply(pos, t), wq)
    flat = torch.empty(T * Hq * D + 1, dtype=torch.bfloat16, device="cuda")
    odd = flat[1:].view(T, Hq, D)
    odd.copy_(q)
    assert torch.equal(rope.apply(pos, odd), wq)
    one = q[:, :1].expand(T, Hq, D)
    assert torch.equal(rope.apply(pos, one), rope.apply(pos, one.contiguous()))
    # every second token
    assert torch.equal(rope.apply(pos[:, ::2].contiguous(), q[::2]), wq[::2])


def test_gradients(aa):
    T, Hq, Hk, D = 45, 4, 2, 64
    rope = aa.RopeAxes(D, (10, 11, 11), base=1e4, interleaved=True)
    theta = [1e4 ** (-2.0 * p / D) for p in range(D // 2)]
    q, k, pos = _data(T, Hq, Hk, D, 3)
    gq, gk, _ = _data(T, Hq, Hk, D, 3, seed=2)
    q.requires_grad_(True), k.requires_grad_(True)
    yq, yk = aa.rope_axes(rope, pos, q, k)
    dq, dk = torch.autograd.grad((yq, yk), (q, k), (gq, gk), create_graph=True)
    _check(dq, gq, pos, rope, theta, False, inverse=True)
    _check(dk, gk, pos, rope, theta, False, inverse=True)
    # differences: L = <gq, rot(q)> is linear in q, so (L(q + d) - L(q)) = <dq, d>, up to the roundings to bf16 of
    # rot(q + d), rot(q) and dq: half a step of each element, 2^-8
    d = torch.randn(q.shape, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    q2 = (q.detach().double() + d.double()).to(torch.bfloat16)
    step = q2.double() - q.detach().double()
    a, b = rope.apply(pos, q2).double(), yq.detach().double()
    lhs, rhs = (gq.double() * (a - b)).sum(), (dq.detach().double() * step).sum()
    room = 2.0 ** -7 * ((gq.double() * a).abs().sum() + (gq.double() * b).abs().sum() + (dq.double() * step).abs().sum())
    assert abs(lhs - rhs) <= room
    # one of the two, q alone, and a k that needs none
    y = aa.rope_axes(rope, pos, q)
    assert torch.equal(torch.autograd.grad(y, q, gq)[0], dq)
    yq, yk = aa.rope_axes(rope, pos, q.detach(), k)
    assert torch.equal(torch.autograd.grad((yq.float().sum() * 0 + yk.float().mul(gk.float()).sum()), k)[0], dk)
    yq, yk = aa.rope_axes(rope, pos, q, k.detach())
    assert torch.equal(torch.autograd.grad(yq, q, gq)[0], dq)


def test_second_derivative_turns_forward(aa):
    rope = aa.RopeAxes(64, (32,), base=1e4)
    q, _, pos = _data(9, 2, 1, 64, 1)
    g = torch.ones_like(q).requires_grad_(True)
    q.requires_grad_(True)
    (dq,) = torch.autograd.grad(aa.rope_axes(rope, pos, q), q, g, create_graph=True)
    v, _, _ = _data(9, 2, 1, 64, 1, seed=4)
    (gg,) = torch.autograd.grad(dq, g, v)
    assert torch.equal(gg, rope.apply(pos, v))


def test_broadcast_inputs_sum_their_gradient(aa):
    rope = aa.RopeAxes(64, (32,), base=1e4)
    _, _, pos = _data(12, 1, 1, 64, 1)
    one = torch.randn(12, 1, 64, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda().requires_grad_(True)
    g, _, _ = _data(12, 4, 1, 64, 1, seed=8)
    aa.rope_axes(rope, pos, one.expand(12, 4, 64)).backward(g)
    want = rope.apply(pos, g, inverse=True).float().sum(1, keepdim=True)
    assert ((one.grad.float() - want).abs() <= 2.0 ** -6 * rope.apply(pos, g, inverse=True).float().abs().sum(1, keepdim=True)).all()


def test_training_step_with_a_plan(aa):
    """Rotation on three axes, then AnchorAttention on a plan that does not rotate: both directions, against the oracle."""
    import oracle as orc
    from gpu_common import REL_L2, f64, inputs, problem, rel_l2
    cu, T, Hq, Hkv, D = [1, 90, 300, 411], 411, 4, 2, 128
    rope = aa.RopeAxes(D, (16, 24, 24), base=5e6)
    theta = [5e6 ** (-2.0 * p / D) for p in range(D // 2)]
    q0, k0, v0, do = inputs(T, Hq, Hkv, D, seed=81)
    _, _, pos = _data(T, 1, 1, D, 3)
    with aa.Plan(cu, T, Hq, Hkv, D, rope_layout=aa.ROPE_NONE) as plan:
        q, k, v = (x.clone().requires_grad_(True) for x in (q0, k0, v0))
        rq, rk = aa.rope_axes(rope, pos, q, k)
        o = aa.anchor_attention(plan, rq, rk, v)
        o.backward(do)
        torch.cuda.synchronize()
        plan.check_device_error()
    prob = problem(cu, T, Hq, Hkv, D, 1e4, layout=orc.ROPE_NONE)
    tq, tk = ref.turn(q0, pos, rope.axis_of_pair, theta, False), ref.turn(k0, pos, rope.axis_of_pair, theta, False)
    O, L = orc.forward(prob, tq.numpy(), tk.numpy(), f64(v0))
    assert abs(f64(o) - O).max() <= 2e-2
    gq, gk, gv = orc.backward(prob, tq.numpy(), tk.numpy(), f64(v0), f64(do))
    gq = ref.turn(torch.from_numpy(gq), pos, rope.axis_of_pair, theta, False, inverse=True).numpy()
    gk = ref.turn(torch.from_numpy(gk), pos, rope.axis_of_pair, theta, False, inverse=True).numpy()
    for name, got, want in (("dq", q.grad, gq), ("dk", k.grad, gk), ("dv", v.grad, gv)):
        assert rel_l2(got, want) <= REL_L2, name


def test_stream_graph_and_refusals(aa):
    T, Hq, Hk, D = 200, 4, 2, 128
    rope = aa.RopeAxes(D, (64,), base=1e4)
    q, k, pos = _data(T, Hq, Hk, D, 1)
    want = rope.apply(pos, q, k)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = rope.apply(pos, q, k, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(q), torch.empty_like(k)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rope.apply(pos, q, k, out_q=out[0], out_k=out[1])
    pos.add_(7)
    graph.replay()
    torch.cuda.synchronize()
    want = rope.apply(pos, q, k)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    assert rope.apply(pos[:, :0].contiguous(), q[:0]).shape == (0, Hq, D)
    for bad in (lambda: rope.apply(pos, q.float()), lambda: rope.apply(pos.long(), q), lambda: rope.apply(pos[:, 1:], q),
                lambda: rope.apply(pos, q, k[1:]), lambda: rope.apply(pos, q[..., :64]), lambda: rope.apply(pos.cpu(), q),
                lambda: rope.apply(pos, q.cpu()), lambda: rope.apply(pos, q, out_k=k),
                lambda: rope.apply(pos, q, out_q=torch.empty_like(q)[:, ::2]), lambda: rope.apply(pos, q, k, out_q=out[0][1:])):
        with pytest.raises(ValueError):
            bad()


def test_empty_calls_with_keys(aa):
    rope = aa.RopeAxes(128, (32, 32), base=1e4)
    q, k, pos = _data(4, 4, 2, 128, 2)
    yq, yk = rope.apply(pos[:, :0].contiguous(), q[:0], k[:0])
    assert yq.shape == (0, 4, 128) and yk.shape == (0, 2, 128)
    q0, k0 = q[:0].clone().requires_grad_(True), k[:0].clone().requires_grad_(True)
    yq, yk = aa.rope_axes(rope, pos[:, :0].contiguous(), q0, k0)
    (yq.sum() + yk.sum()).backward()
    assert q0.grad.shape == (0, 4, 128) and k0.grad.shape == (0, 2, 128)


def test_results_written_into_given_tensors_are_seen_by_autograd(aa):
    """A result tensor is a written tensor: a graph that saved its old values says so, and one that would carry a wrong
    gradient is refused."""
    rope = aa.RopeAxes(64, (32,), base=1e4)
    x, _, pos = _data(9, 2, 1, 64, 1)
    x.requires_grad_(True)
    a = x * 2
    y = a * a  # saves a
    for out in (a, x):
        with pytest.raises(ValueError, match="grad"):
            rope.apply(pos, a.detach().clone(), out_q=out)
    y.float().sum().backward(retain_graph=True)  # refused calls have written nothing
    with torch.no_grad():
        rope.apply(pos, a, out_q=a)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.float().sum().backward()
    with torch.inference_mode():
        z = torch.zeros_like(a)
    assert torch.equal(rope.apply(pos, a.detach(), out_q=z), rope.apply(pos, a.detach()))


def test_training_step_in_a_graph(aa):
    """Forward and gradient captured after a warm-up on a side stream, whose autograd graph is gone by then (PyTorch ties
    the leaves of a living one to the stream that it was made on, and refuses the capture)."""
    T, Hq, Hk, D = 64, 4, 2, 64
    rope = aa.RopeAxes(D, (32,), base=1e4)
    q, k, pos = _data(T, Hq, Hk, D, 1)
    gq, gk, _ = _data(T, Hq, Hk, D, 1, seed=2)
    q.requires_grad_(True), k.requires_grad_(True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = torch.autograd.grad(aa.rope_axes(rope, pos, q, k), (q, k), (gq, gk))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = torch.autograd.grad(aa.rope_axes(rope, pos, q, k), (q, k), (gq, gk))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
