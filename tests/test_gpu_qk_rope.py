"""Norms and rotation of queries and keys on the GPU, forward and backward,
against the plain 64-bit forms of kv_reference.py.

Bounds: a result is rounded to bf16 once (half a step, HALF_STEP relative); what
comes before is FP32 on magnitudes up to `size` (the pair's or the row's), with
the table's own FP32 rounding and a few tens of operations: 2^-18 of it."""
import numpy as np
import pytest
import torch

import kv_reference as R
from bit_attention_gb300 import qk_rope as Q
from bit_attention_gb300 import sage_fp4 as S

pytestmark = pytest.mark.gpu
F32_SLACK = 2.0 ** -18


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16).cuda()


def close(got, ref, size, what):
    d = np.abs(R.f64(got) - ref)
    tol = R.HALF_STEP * np.abs(ref) + F32_SLACK * size + 1e-37
    assert (d <= tol).all(), (what, float((d / tol).max()))


def case(seed, B, N, Hq, Hk, D, norm=True, wdtype=torch.float32):
    rng = np.random.default_rng(seed)
    x = bf16(1.5 * rng.standard_normal((B, N, Hq + 2 * Hk, D)))
    x[:, ::5, 0] *= 1e-3
    w = [torch.from_numpy(1 + 0.3 * rng.standard_normal(D)).to(wdtype).cuda() if norm else None for _ in range(2)]
    return rng, x[:, :, :Hq], x[:, :, Hq:Hq + Hk], w


def reference(x, w, pos, rot, inter, g=None, **angles):
    cos, sin = R.rope_angles(pos, rot, **angles)
    w = None if w is None else R.f64(w)
    y = R.rope(R.f64(x), cos, sin, rot, inter, w)
    return (y, None, None) if g is None else (y, *R.rope_back(R.f64(x), R.f64(g), cos, sin, rot, inter, w))


@pytest.mark.parametrize("B,N,Hq,Hk,D,rot", [(1, 1, 1, 1, 64, 64), (2, 37, 12, 4, 64, 32), (1, 300, 32, 8, 128, 128),
                                            (3, 5, 7, 1, 128, 48), (1, 2000, 9, 3, 64, 16), (1, 65, 5, 5, 128, 96)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_forward_and_backward_match_the_formulas(B, N, Hq, Hk, D, rot, inter, norm):
    rng, q, k, w = case(N + D, B, N, Hq, Hk, D, norm, torch.bfloat16 if N % 2 else torch.float32)
    pos = rng.integers(0, 5000, (B, N))
    table = Q.rope_table(5000, rot)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    gq, gk = (bf16(0.01 * rng.standard_normal((B, h, N, D))) for h in (Hq, Hk))
    yq, yk = Q.forward(q, k, p, table, *w, interleaved=inter, out_layout="HND")
    back = Q.backward(gq, gk, q, k, p, table, *w, interleaved=inter, grad_layout="HND")
    assert table.get_status() == S.OK
    for x, wx, y, g, dx, dw in ((q, w[0], yq, gq, back[0], back[2]), (k, w[1], yk, gk, back[1], back[3])):
        ry, rdx, rdw = reference(x, wx, pos, rot, inter, g.transpose(1, 2))
        close(y.transpose(1, 2), ry, np.abs(ry).max(-1, keepdims=True) * 2, "y")
        # dx: the two terms of a row are of the size of r * max |g w|
        size = 1.0 if wx is None else np.abs(R.f64(wx)).max() / np.sqrt((R.f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
        close(dx, rdx, size * np.abs(R.f64(g.transpose(1, 2))).max(-1, keepdims=True) * 8, "dx")
        if norm:
            # FP32 sums of the rows' terms, at most 2^-24 of the terms' magnitudes an addition and 2^-20 a term
            cos, sin = R.rope_angles(pos, rot)
            t, _ = R.rope_back(R.f64(x), R.f64(g.transpose(1, 2)), cos, sin, rot, inter)
            xh = R.f64(x) / np.sqrt((R.f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
            a = np.abs(R.f64(g)).max() * 1.5 * np.abs(xh).reshape(-1, D).sum(0)
            rows = B * N * x.shape[2]
            assert (np.abs(R.f64(dw) - rdw) <= a * (2.0 ** -20 + 2.0 ** -24 * (rows ** 0.5 + 16))).all()
        else:
            assert dw is None


@pytest.mark.parametrize("scaling", [dict(), dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=8.0, trained=4096)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_far_positions_and_scaled_tables(scaling, base):
    # positions up to 2^20: the angles are made in 64 bits, so they lose nothing
    rng, q, k, w = case(3, 1, 64, 4, 2, 128)
    n = 1 << 20
    pos = np.concatenate([np.arange(n - 32, n), rng.integers(0, n, 32)])[None]
    table = Q.rope_table(n, 128, base=base, **scaling)
    y, _ = Q.forward(q, k, torch.from_numpy(pos.astype(np.int32)).cuda(), table, *w)
    ry, _, _ = reference(q, w[0], pos, 128, False, base=base, **scaling)
    close(y, ry, np.abs(ry).max(-1, keepdims=True) * 2, "y")


def test_layouts_strides_in_place_and_positions():
    rng, q, k, w = case(5, 2, 33, 6, 2, 64)
    table = Q.rope_table(100, 64)
    p1 = torch.arange(33, dtype=torch.int32, device="cuda")
    ref = Q.forward(q.contiguous(), k.contiguous(), p1, table, *w)
    same = lambda got, r=ref: all(torch.equal(a, b) for a, b in zip(got, r))  # noqa: E731
    assert same(Q.forward(q, k, p1, table, *w))
    assert same(Q.forward(q, k, p1.expand(2, 33).contiguous(), table, *w))
    hnd = Q.forward(q.transpose(1, 2), k.transpose(1, 2), p1, table, *w, layout="HND")
    assert same([x.transpose(1, 2) for x in hnd])
    assert same(Q.forward(q.transpose(1, 2), k.transpose(1, 2), p1, table, *w, layout="HND", out_layout="NHD"))
    flat = Q.forward(q[0], k[0], p1, table, *w)  # packed [tokens, H, D]
    assert same(flat, [x[0] for x in ref])
    whole = torch.cat([q, k], 2)
    rest = whole.clone()
    q2, k2 = whole[:, :, :6], whole[:, :, 6:]
    assert same(Q.forward(q2, k2, p1, table, *w, out=(q2, k2)))  # in place, in a packed tensor
    assert torch.equal(torch.cat(ref, 2), whole) and not torch.equal(rest, whole)
    one = q[:, :1].expand(2, 33, 6, 64)  # a broadcast input
    assert same(Q.forward(one, k, p1, table, *w), Q.forward(one.contiguous(), k, p1, table, *w))
    gq, gk = (torch.ones((), dtype=torch.bfloat16, device="cuda").expand(x.shape) for x in (q, k))
    a = Q.backward(gq, gk, q, k, p1, table, *w)
    c = Q.backward(gq.contiguous(), gk.contiguous(), q, k, p1, table, *w)
    assert all(torch.equal(x, y) for x, y in zip(a, c))


@pytest.mark.parametrize("bad", [-1, 100, 2 ** 31 - 1, -2 ** 31])
def test_a_position_outside_the_table_is_recorded_and_left_out(bad):
    rng, q, k, w = case(6, 1, 20, 3, 2, 64)
    table = Q.rope_table(100, 32)
    p = torch.arange(20, dtype=torch.int32, device="cuda")
    pb = p.clone()
    pb[7] = bad
    live = [i for i in range(20) if i != 7]
    gq, gk = torch.randn_like(q), torch.randn_like(k)
    gz = [g.clone() for g in (gq, gk)]
    for g in gz:
        g[:, 7] = 0
    ref, rb = Q.forward(q, k, p, table, *w), Q.backward(*gz, q, k, p, table, *w)
    assert table.get_status() == S.OK
    got = Q.forward(q, k, pb, table, *w)
    assert table.get_status() == S.EINDEX and table.get_status() == S.OK
    gb = Q.backward(gq, gk, q, k, pb, table, *w)
    assert table.get_status() == S.EINDEX
    for a, b in zip(got + gb[:2], ref + rb[:2]):
        assert (a[:, 7] == 0).all() and torch.equal(a[:, live], b[:, live])
    assert torch.equal(gb[2], rb[2]) and torch.equal(gb[3], rb[3])


def test_autograd_matches_differences_and_casts_the_weights_gradients():
    # directional derivatives of sum(c * y) in 64 bits against the autograd result
    B, N, Hq, Hk, D, rot = 2, 9, 4, 2, 64, 32
    for wdtype in (torch.float32, torch.bfloat16):
        rng, q, k, w = case(8, B, N, Hq, Hk, D, True, wdtype)
        pos = np.arange(N)[None].repeat(B, 0)
        table = Q.rope_table(64, rot)
        leaves = [x.detach().clone().requires_grad_() for x in (q, k, *w)]
        p = torch.arange(N, dtype=torch.int32, device="cuda")
        y = Q.norm_rope(leaves[0], leaves[1], p, table, leaves[2], leaves[3], interleaved=True)
        c = [bf16(rng.standard_normal(x.shape)) for x in y]
        grads = torch.autograd.grad(y, leaves, c)
        assert [g.dtype for g in grads] == [x.dtype for x in leaves] and [g.shape for g in grads] == [x.shape for x in leaves]
        for i in range(2):
            x0, w0, c0 = R.f64(leaves[i]), R.f64(leaves[2 + i]), R.f64(c[i])
            f = lambda x, ww: (reference_y(x, ww, pos, rot) * c0).sum()  # noqa: E731
            dx, dw = rng.standard_normal(x0.shape), rng.standard_normal(D)
            h = 1e-5
            num_x, num_w = (f(x0 + h * dx, w0) - f(x0 - h * dx, w0)) / (2 * h), (f(x0, w0 + h * dw) - f(x0, w0 - h * dw)) / (2 * h)
            gx, gw = R.f64(grads[i]), R.f64(grads[2 + i])
            # each gradient element is rounded to its type: half a step; the differences' own error is below 1e-6 here
            assert abs((gx * dx).sum() - num_x) <= (R.HALF_STEP * 1.1 * np.abs(gx * dx)).sum() + 1e-4
            step = R.HALF_STEP if wdtype == torch.bfloat16 else 2.0 ** -18
            assert abs((gw * dw).sum() - num_w) <= (step * 1.1 * np.abs(gw * dw)).sum() + 1e-3


def reference_y(x, w, pos, rot):
    cos, sin = R.rope_angles(pos, rot)
    return R.rope(x, cos, sin, rot, True, w)


def test_without_gradients_nothing_is_kept_and_one_sided_gradients_work():
    rng, q, k, w = case(9, 1, 5, 2, 2, 64)
    table = Q.rope_table(8, 64)
    p = torch.arange(5, dtype=torch.int32, device="cuda")
    assert all(x.grad_fn is None for x in Q.norm_rope(q, k, p, table, *w))
    leaf = q.detach().clone().requires_grad_()
    y = Q.norm_rope(leaf, k, p, table, *w)
    y[1].float().sum().backward()  # nothing flows to q's result
    assert (leaf.grad == 0).all()
    with torch.no_grad():
        assert Q.norm_rope(leaf, k, p, table, *w)[0].grad_fn is None
    y = Q.norm_rope(leaf, k, p, table, *w)
    with pytest.raises(RuntimeError):  # no second derivatives
        g, = torch.autograd.grad(y[0].float().sum(), leaf, create_graph=True)
        torch.autograd.grad(g.float().sum(), leaf)


def test_saved_tensors_that_hooks_move_or_lay_out_anew():
    # hooks that keep a copy elsewhere, and ones that bring it back to the same
    # address with other strides
    rng, q, k, w = case(12, 1, 40, 4, 2, 64)
    table = Q.rope_table(64, 64)
    p = torch.arange(40, dtype=torch.int32, device="cuda")
    g = [torch.randn(x.shape, device="cuda").to(torch.bfloat16) for x in (q, k)]

    def grads(pack, unpack):
        wide, own = torch.cat([q, k], 2).requires_grad_(), k.clone().requires_grad_()
        with torch.autograd.graph.saved_tensors_hooks(pack, unpack):
            y = Q.norm_rope(wide[:, :, :4], own, p, table, *w)
        return torch.cat([x.flatten() for x in torch.autograd.grad(y, (wide, own), g)])

    ref = grads(lambda t: t, lambda t: t)

    def densely(t):
        with torch.no_grad():
            if t.dtype != torch.bfloat16 or t.dim() != 4 or t.shape[2] != 4:
                return t
            copy = t.contiguous()
            room = t.as_strided((t.numel(),), (1,))  # from the tensor's own address on
            return copy, room

    def back(t):
        if isinstance(t, torch.Tensor):
            return t
        with torch.no_grad():
            copy, room = t
            room.copy_(copy.flatten())
            return room.view(copy.shape)

    assert torch.equal(grads(densely, back), ref)
    assert torch.equal(grads(lambda t: t.cpu(), lambda t: t.cuda()), ref)


def test_misfits_are_refused():
    rng, q, k, w = case(13, 1, 12, 4, 2, 64)
    q, k = q.contiguous(), k.contiguous()
    table = Q.rope_table(64, 64)
    p = torch.arange(12, dtype=torch.int32, device="cuda")
    shared = torch.empty_like(q[:, :1]).expand(q.shape)
    for call in (lambda: Q.forward(q, k, p, table, *w, out=(shared, k)), lambda: Q.forward(q, k, p, table, *w, out=(k, q)),
                 lambda: Q.forward(q, k[:, :11], p, table, *w), lambda: Q.forward(q, k, p.long(), table, *w),
                 lambda: Q.forward(q, k, p[:11], table, *w), lambda: Q.forward(q, k, p.cpu(), table, *w),
                 lambda: Q.forward(q, k, p, table, w[0], w[1].bfloat16()), lambda: Q.forward(q, k, p, table, w[0]),
                 lambda: Q.forward(q, k, p, table, w[0][:32], w[1]), lambda: Q.forward(q.float(), k, p, table, *w),
                 lambda: Q.forward(q, k, p, Q.rope_table(64, 128), *w), lambda: Q.forward(q, k, p, table, *w, eps=-1.0),
                 lambda: Q.forward(q, k, p, table, *w, layout="BNHD"), lambda: Q.forward(q[0], k[0], p, table, *w, layout="HND"),
                 lambda: Q.forward(q[..., ::2], k[..., ::2], p, table), lambda: Q.forward(q.flatten()[4:260].view(1, 1, 4, 64), k[:, :1], p[:1], table, *w),
                 lambda: Q.backward(q[:, :11], k, q, k, p, table, *w), lambda: Q.backward(q.float(), k, q, k, p, table, *w),
                 lambda: Q.backward(q, k, q, k, p, table, *w, grad_layout="BNHD")):
        with pytest.raises(S.SageFp4Error) as e:
            call()
        assert e.value.code == S.EINVAL
    assert table.get_status() == S.OK


def test_empty_problems():
    w = [torch.ones(64, device="cuda") for _ in range(2)]
    table = Q.rope_table(8, 64)
    for B, N, Hq, Hk in ((0, 4, 2, 2), (2, 0, 2, 2), (1, 3, 0, 0)):
        q, k = (torch.empty((B, N, h, 64), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hk))
        p = torch.zeros(N, dtype=torch.int32, device="cuda")
        y = Q.forward(q.as_strided(q.shape, (0, 0, 0, 0)) if q.numel() == 0 else q, k, p, table, *w)
        assert y[0].shape == q.shape
        dq, dk, dwq, dwk = Q.backward(y[0], y[1], q, k, p, table, *w)
        assert dq.shape == q.shape and (dwq == 0).all() and (dwk == 0).all()
    assert table.get_status() == S.OK


def test_replays_from_a_graph_and_runs_on_another_stream():
    rng, q, k, w = case(10, 1, 50, 8, 2, 128)
    table = Q.rope_table(4096, 128)
    q, k = q.contiguous(), k.contiguous()
    p = torch.arange(50, dtype=torch.int32, device="cuda")
    gq, gk = torch.randn_like(q), torch.randn_like(k)

    def step():
        return Q.forward(q, k, p, table, *w) + Q.backward(gq, gk, q, k, p, table, *w)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(3):
        p.copy_(torch.arange(50, dtype=torch.int32, device="cuda") + 100 * i)
        q.copy_(torch.randn_like(q))
        g.replay()
        ref = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, ref))
    side = torch.cuda.Stream()
    torch.cuda._sleep(2_000_000)
    q2 = q * 1.0
    y = Q.forward(q2, k, p, table, *w, stream=side)
    b = Q.backward(gq, gk, q2, k, p, table, *w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, c) for a, c in zip(y + b, ref))


@pytest.mark.parametrize("wdtype", [torch.float32, torch.bfloat16])
def test_a_captured_training_step(wdtype):
    # forward and autograd's backward in one graph, warmed up on the capturing
    # stream and with no other graph of the leaves alive
    rng, q, k, w = case(14, 1, 70, 4, 2, 64, True, wdtype)
    table = Q.rope_table(128, 64)
    p = torch.arange(70, dtype=torch.int32, device="cuda")
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, *w)]
    g = [torch.randn_like(x) for x in leaves[:2]]

    def step():
        return torch.autograd.grad(Q.norm_rope(leaves[0], leaves[1], p, table, *leaves[2:]), leaves, g)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = step()
    for i in range(3):
        with torch.no_grad():
            for x in leaves[:2] + g:
                x.copy_(torch.randn_like(x))
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
    assert table.get_status() == S.OK


def test_the_rotation_in_front_of_sagebwd_trains():
    # q and k through norm_rope into the 8-bit training attention and back
    from bit_attention_gb300 import sagebwd as SB
    rng, q, k, w = case(11, 1, 256, 2, 2, 64)
    v = bf16(rng.standard_normal((1, 2, 256, 64))).requires_grad_()
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, *w)]
    table = Q.rope_table(256, 64)
    p = torch.arange(256, dtype=torch.int32, device="cuda")
    y = Q.norm_rope(leaves[0], leaves[1], p, table, leaves[2], leaves[3], out_layout="HND")
    o = SB.attention(*y, v, causal=True)
    o.backward(torch.randn_like(o))
    y2 = [x.detach().requires_grad_() for x in y]
    assert all(torch.isfinite(x.grad).all() and (x.grad != 0).any() for x in leaves)
    # the same gradients as through the two backward calls by hand
    o2 = SB.attention(*y2, v.detach(), causal=True)
    assert torch.equal(o2, o)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hk", [(12, 4), (8, 8), (9, 1), (32, 16)])
@pytest.mark.parametrize("inter", [False, True])
def test_an_eps_of_zero_and_heads_that_leave_a_rest(D, Hq, Hk, inter):
    # heads that do not fill a warp's unit, and a token left out whose rows are zeros
    B, N, rot = 2, 21, 48
    rng, q, k, w = case(15, B, N, Hq, Hk, D)
    q[1, 3], k[1, 3] = 0.0, 0.0
    pos = rng.integers(0, 500, (B, N))
    pos[1, 3] = 500
    live = (pos < 500).reshape(-1)
    table = Q.rope_table(500, rot)
    p = torch.from_numpy(pos.astype(np.int32)).cuda()
    gq, gk = (bf16(0.01 * rng.standard_normal((B, N, h, D))) for h in (Hq, Hk))
    y = Q.forward(q, k, p, table, *w, eps=0.0, interleaved=inter)
    back = Q.backward(gq, gk, q, k, p, table, *w, eps=0.0, interleaved=inter)
    assert table.get_status() == S.EINDEX
    cos, sin = (x.reshape(B * N, -1)[live] for x in R.rope_angles(pos, rot))
    for x, wx, got, g, dx, dw in ((q, w[0], y[0], gq, back[0], back[2]), (k, w[1], y[1], gk, back[1], back[3])):
        x, g = (R.f64(t).reshape(B * N, -1, D)[live] for t in (x, g))
        rms, wx = np.sqrt((x * x).mean(-1, keepdims=True)), R.f64(wx)
        ry, (rdx, rdw) = R.rope(x, cos, sin, rot, inter, wx, 0.0), R.rope_back(x, g, cos, sin, rot, inter, wx, 0.0)
        got, dx = (t.reshape(B * N, -1, D) for t in (got, dx))
        on = torch.from_numpy(live)
        close(got.cpu()[on], ry, np.abs(ry).max(-1, keepdims=True) * 2, "y")
        close(dx.cpu()[on], rdx, np.abs(wx).max() / rms * np.abs(g).max(-1, keepdims=True) * 8, "dx")
        assert (got.cpu()[~on] == 0).all() and (dx.cpu()[~on] == 0).all()
        a = np.abs(g).max() * 1.5 * np.abs(x / rms).reshape(-1, D).sum(0)
        assert (np.abs(R.f64(dw) - rdw) <= a * (2.0 ** -20 + 2.0 ** -24 * (x.shape[0] * x.shape[1]) ** 0.5 + 2.0 ** -20)).all()


def test_forward_mode_is_refused():
    import torch.autograd.forward_ad as F
    rng, q, k, w = case(16, 1, 6, 2, 2, 64)
    table = Q.rope_table(8, 64)
    p = torch.arange(6, dtype=torch.int32, device="cuda")
    ref = Q.norm_rope(q, k, p, table, *w)
    with F.dual_level():  # no input has a tangent
        assert all(torch.equal(a, b) for a, b in zip(Q.norm_rope(q, k, p, table, *w), ref))
    for i in range(4):
        with F.dual_level():
            x = [q, k, *w]
            x[i] = F.make_dual(x[i], torch.ones_like(x[i]))
            with pytest.raises(NotImplementedError):
                Q.norm_rope(x[0], x[1], p, table, x[2], x[3])
            with torch.no_grad(), pytest.raises(NotImplementedError):
                Q.norm_rope(x[0], x[1], p, table, x[2], x[3])
    with pytest.raises(RuntimeError):
        torch.func.jvp(lambda x: Q.norm_rope(x, k, p, table, *w)[0], (q.contiguous(),), (torch.ones_like(q),))


def test_a_status_is_read_on_its_own_stream():
    # while the default stream is busy with something else
    table = Q.rope_table(8, 64)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    table.status[0] = S.EINDEX
    torch.cuda.synchronize()
    torch.cuda._sleep(500_000_000)
    assert table.get_status(side) == S.EINDEX and table.get_status(side) == S.OK
    assert not torch.cuda.current_stream().query()


def test_gradients_through_sagebwd_are_those_of_the_calls_by_hand():
    # autograd through norm_rope and the 8-bit attention against both backward calls
    from bit_attention_gb300 import sagebwd as SB
    rng, q, k, w = case(17, 1, 256, 2, 2, 64)
    v = bf16(rng.standard_normal((1, 2, 256, 64))).requires_grad_()
    leaves = [x.detach().clone().requires_grad_() for x in (q, k, *w)]
    table = Q.rope_table(256, 64)
    p = torch.arange(256, dtype=torch.int32, device="cuda")
    o = SB.attention(*Q.norm_rope(leaves[0], leaves[1], p, table, leaves[2], leaves[3], out_layout="HND"), v, causal=True)
    do = torch.randn_like(o)
    o.backward(do)
    y = [x.detach().requires_grad_() for x in Q.forward(q, k, p, table, *w, out_layout="HND")]
    SB.attention(*y, v.detach(), causal=True).backward(do)
    by_hand = Q.backward(y[0].grad, y[1].grad, q, k, p, table, *w, grad_layout="HND")
    assert all(torch.equal(x.grad, g) for x, g in zip(leaves, by_hand))


def test_results_laid_over_inputs_other_than_in_place_are_refused():
    rng, q, k, w = case(18, 2, 9, 4, 4, 64)
    q, k = q.contiguous(), k.contiguous()
    table = Q.rope_table(64, 64)
    p = torch.arange(9, dtype=torch.int32, device="cuda")
    fresh = [torch.empty_like(x) for x in (q, k)]
    anew = q.view(2, 4, 9, 64)  # q's memory as [B, H, N, D]
    keep = [q.clone(), k.clone()]
    for out, layout in (((k, q), "NHD"), ((fresh[0], fresh[0]), "NHD"), ((k, fresh[1]), "NHD"), ((fresh[0], q), "NHD"),
                        ((anew, torch.empty_like(anew)), "HND")):
        with pytest.raises(S.SageFp4Error) as e:
            Q.forward(q, k, p, table, *w, out=out, out_layout=layout)
        assert e.value.code == S.EINVAL
    assert torch.equal(q, keep[0]) and torch.equal(k, keep[1]) and table.get_status() == S.OK
    ref = Q.forward(q, k, p, table, *w)
    Q.forward(q, k, p, table, *w, out=(fresh[0], k))  # one of the two in place
    assert torch.equal(fresh[0], ref[0]) and torch.equal(k, ref[1])
