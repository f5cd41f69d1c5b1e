"""The operators around the scan as a Mamba block uses them: prompts and tokens of a Mamba-2
block, the training of a Mamba-1 block, captured and replayed graphs, other streams, both ways
of marshalling a call, and the binding's refusals.

A chain of calls is checked stage by stage: each stage's float64 oracle takes what the GPU's
stage before it gave, so that every bar is that stage's own.
"""
import numpy as np
import pytest

import oracle
import selective_state_space_fwd_amd as ssm
from block_util import TOL, Rand, check, same, sum_tol
from gpu_util import announce, dev, host, torch
from oracle import block as ob
from ssm_workloads import RTOL, RTOL_STATE, WATCH
from test_gpu_graph import unrelated_eager_work
from test_gpu_norm import grad_tol

pytestmark = pytest.mark.gpu

HEADS, P, N, W = 4, 32, 64, 4
D = HEADS * P
WIDE = D + D + 2 * N + HEADS          # a projection's output: z, x, B, C, dt


class Block:
    """A Mamba-2 block between its projections."""

    def __init__(self, seed):
        r = Rand(seed)
        self.w, self.bias = r((D + 2 * N, W), scale=0.5), r((D + 2 * N,), scale=0.5)
        self.A = torch().tensor([-1.0, -2.0, -4.0, -8.0], device="cuda")
        self.dt_bias, self.D, self.nw = r((HEADS,)), r((D,)), r((D,))

    def cut(self, proj):
        return proj[..., :D], proj[..., D:2 * D + 2 * N], proj[..., 2 * D + 2 * N:]

    def prompt(self, proj, lengths=None, conv_state=None, h0=None):
        """proj: [batch, seqlen, WIDE]. Returns every stage's result."""
        z, xbc, dt = (v.transpose(1, 2) for v in self.cut(proj))
        u, cs = ssm.conv(xbc, self.w[0], bias=self.bias[0], silu=True, lengths=lengths,
                         initial_state=conv_state)
        mask = None
        if lengths is not None:
            mask = torch().arange(proj.shape[1], device="cuda")[None] < lengths[:, None]
        y, h = ssm.ssd(u[:, :D], dt.contiguous(), self.A, u[:, D:D + N], u[:, D + N:], D=self.D[0],
                       dt_bias=self.dt_bias[0], dt_softplus=True, mask=mask, h0=h0)
        return u, cs, y, h, ssm.norm(y, self.nw[0], z=z, token_major=True)

    def token(self, proj, conv_cache, cache, slots, outs=(None, None, None)):
        """proj: [batch, WIDE]."""
        z, xbc, dt = self.cut(proj)
        u = ssm.conv_step(xbc, conv_cache, self.w[0], bias=self.bias[0], silu=True, slots=slots,
                          out=outs[0])
        y = ssm.ssd_step(u[:, :D], dt, self.A, u[:, D:D + N], u[:, D + N:], cache, D=self.D[0],
                         dt_bias=self.dt_bias[0], dt_softplus=True, slots=slots, out=outs[1])
        return u, y, ssm.norm(y[:, :, None], self.nw[0], z=z[:, :, None], token_major=True,
                              out=outs[2])


def test_mamba2_block_prompt_then_tokens():
    """A padded bucket of prompts, their states put into slots of the caches, then tokens of all
    of them; every stage against its oracle, and the tokens against the same tokens taken as
    the end of a longer prompt."""
    announce("mamba-2 block: prompt, then tokens")
    t = torch()
    m, r = Block(700), Rand(701)
    b, L, steps, slots_n = 3, 90, 5, 8
    proj = r((b, L + steps, WIDE), "bf16")[0]
    n = [90, 41, 2]
    lengths = t.tensor(n, dtype=t.int32, device="cuda")
    u, cs, y, h, out = m.prompt(proj[:, :L], lengths)
    z, xbc, dt = (host(v).transpose(0, 2, 1) for v in m.cut(proj[:, :L].contiguous()))
    live = np.arange(L)[None] < np.array(n)[:, None]
    ref, rcs = ob.conv_ref(xbc, m.w[1], m.bias[1], True, lengths=n)
    check(u, ref, TOL["bf16"], "conv")
    assert np.array_equal(host(cs), rcs)
    uh = host(u)
    ref, rh = oracle.ssd_ref(uh[:, :D], dt, host(m.A), uh[:, D:D + N], uh[:, D + N:], m.D[1], None,
                             m.dt_bias[1], True, None, mask=live.astype(np.uint8))
    check(y, ref, RTOL["bf16"], "ssd")
    check(h, rh, RTOL_STATE, "ssd state")
    check(out, ob.norm_ref(host(y), m.nw[1], z)[0].transpose(0, 2, 1), TOL["bf16"], "norm")

    slots = t.tensor([6, 0, 3], dtype=t.int32, device="cuda")
    conv_cache = t.full((slots_n, D + 2 * N, W - 1), 7.0, device="cuda", dtype=t.bfloat16)
    cache = t.full((slots_n, D, N), 7.0, device="cuda")
    conv_cache[slots.long()], cache[slots.long()] = cs, h
    got = []
    for s in range(steps):
        p = proj[:, L + s]
        state64, conv64 = host(cache), host(conv_cache)
        u, y, o = m.token(p, conv_cache, cache, slots)
        z, xbc, dt = (host(v) for v in m.cut(p.contiguous()))
        ref, after = ob.conv_step_ref(xbc, conv64, m.w[1], m.bias[1], True, slots.tolist())
        check(u, ref, TOL["bf16"], f"token {s} conv")
        assert np.array_equal(host(conv_cache), after)
        uh = host(u)
        ref, after = ob.step_ref(uh[:, :D], dt, host(m.A), uh[:, D:D + N], uh[:, D + N:], state64,
                                 m.D[1], None, m.dt_bias[1], True, slots.tolist())
        check(y, ref, WATCH["bf16"], f"token {s} state step")
        check(cache, after, 1e-5, f"token {s} state")
        check(o, ob.norm_ref(host(y)[:, :, None], m.nw[1], z[:, :, None])[0].transpose(0, 2, 1),
              TOL["bf16"], f"token {s} norm")
        got.append(o[:, 0])
    # The first row was whole: its tokens continue it, and are the end of a longer prompt. Both
    # ways are within the ssd's bar of the exact value at y, which the norm keeps relative to a
    # token's rms; the rest is roundings to bf16 (three stages, two ways).
    whole = m.prompt(proj[:1])[4]
    got = t.stack([g[0] for g in got])
    check(got, host(whole[0, L:]), 2 * RTOL["bf16"] + 6 * WATCH["bf16"], "tokens, prompt")


def test_mamba2_prompt_in_chunks():
    """A prompt taken in two calls, with the states handed on, is the prompt taken in one."""
    announce("mamba-2 block: prompt in chunks")
    m, r = Block(710), Rand(711)
    proj = r((2, 150, WIDE), "bf16")[0]
    u, cs, y, h, out = m.prompt(proj)
    u1, cs1, y1, h1, out1 = m.prompt(proj[:, :67])
    u2, cs2, y2, h2, out2 = m.prompt(proj[:, 67:], conv_state=cs1, h0=h1)
    t = torch()
    assert same(t.cat((u1, u2), 2), u) and same(cs2, cs)
    check(h2, host(h), 2 * RTOL_STATE, "state")
    check(t.cat((out1, out2), 1), host(out), 2 * RTOL["bf16"] + 4 * WATCH["bf16"], "out")


def test_mamba1_block_training():
    """causal_conv, selective_scan and gated_norm under autograd, fp32, channel-ordered inputs:
    every gradient against the chain of the float64 backward oracles. Each stage is within
    1e-4 of the metric (the scan's bar); three stages in a row, whose gains on random data are
    of order one: 1e-3."""
    announce("mamba-1 block training")
    t = torch()
    r = Rand(720)
    b, d, n, L = 2, 24, 16, 300
    proj, proj64 = r((b, L, 2 * d))
    w, w64 = r((d, 4), scale=0.5)
    bias, bias64 = r((d,), scale=0.5)
    delta, delta64 = r((b, d, L), scale=0.5)
    B, B64 = r((b, n, L), scale=0.5)
    C, C64 = r((b, n, L), scale=0.5)
    A = -t.arange(1, n + 1, device="cuda").float().repeat(d, 1)
    Dk, D64 = r((d,))
    dtb = t.full((d,), -2.0, device="cuda")
    nw, nw64 = r((d,))
    g, g64 = r((b, L, d))
    leaves = [v.requires_grad_() for v in (proj, w, bias, delta, B, C, A, Dk, dtb, nw)]
    x, z = (v.transpose(1, 2) for v in (proj[..., :d], proj[..., d:]))
    u, _ = ssm.causal_conv(x, w, bias, True)
    y, _ = ssm.selective_scan(u, delta, A, B, C, D=Dk, delta_bias=dtb, delta_softplus=True)
    out = ssm.gated_norm(y, nw, z=z, token_major=True)
    (out * g).sum().backward()

    x64, z64 = (np.ascontiguousarray(v.transpose(0, 2, 1)) for v in (proj64[..., :d], proj64[..., d:]))
    A64, dtb64 = host(A), host(dtb)
    u64, _ = ob.conv_ref(x64, w64, bias64, True)
    y64, _ = oracle.scan_ref(u64, delta64, A64, B64, C64, D64, None, dtb64, True)
    out64, _ = ob.norm_ref(y64, nw64, z64)
    check(out, out64.transpose(0, 2, 1), 1e-3, "out")
    gn = ob.norm_bwd_ref(y64, nw64, g64.transpose(0, 2, 1), z64)
    gs = oracle.scan_bwd_ref(u64, delta64, A64, B64, C64, D64, None, dtb64, True, None, gn["dy"], None)
    gc = ob.conv_bwd_ref(x64, w64, gs["du"], bias64, True)
    want = {"x": gc["dx"].transpose(0, 2, 1), "z": gn["dz"].transpose(0, 2, 1), "w": gc["dweight"],
            "bias": gc["dbias"], "delta": gs["ddelta"], "B": gs["dB"], "C": gs["dC"],
            "A": gs["dA"], "D": gs["dD"], "dt_bias": gs["dbias"], "norm": gn["dweight"]}
    have = {"x": proj.grad[..., :d], "z": proj.grad[..., d:], "w": w.grad, "bias": bias.grad,
            "delta": delta.grad, "B": B.grad, "C": C.grad, "A": A.grad, "D": Dk.grad,
            "dt_bias": dtb.grad, "norm": nw.grad}
    for k in want:
        check(have[k], want[k], 1e-3, "d" + k)


# ---------------------------------------------------------------- graphs and streams

def capture(t, work):
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        work()
    t.cuda.current_stream().wait_stream(side)
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        result = work()
    return graph, result


def test_graph_of_tokens():
    """Several tokens of a block captured once, with a padding row of no slot; replayed with new
    projections and slots written into its buffers, against the same calls made eagerly."""
    announce("graph of tokens")
    t = torch()
    m, r = Block(730), Rand(731)
    b, steps, slots_n = 4, 3, 6
    proj = [t.empty((b, WIDE), device="cuda", dtype=t.bfloat16) for _ in range(steps)]
    slots = t.tensor([0, 1, 2, -1], dtype=t.int32, device="cuda")
    conv_cache = t.zeros((slots_n, D + 2 * N, W - 1), device="cuda", dtype=t.bfloat16)
    cache = t.zeros((slots_n, D, N), device="cuda")
    for p in proj:
        p.copy_(r((b, WIDE), "bf16")[0])
    graph, outs = capture(t, lambda: [m.token(p, conv_cache, cache, slots)[2] for p in proj])
    for replay, s in enumerate(([0, 1, 2, -1], [5, 3, 0, 1], [2, -1, -1, 4], [1, 1, 3, 3])):
        new = [r((b, WIDE), "bf16")[0] for _ in range(steps)]
        start_conv, start = r(tuple(conv_cache.shape), "bf16")[0], r(tuple(cache.shape))[0]
        eager_conv, eager = start_conv.clone(), start.clone()
        want_slots = t.tensor(s, dtype=t.int32, device="cuda")
        want = [m.token(p, eager_conv, eager, want_slots)[2] for p in new]
        for dst, src in zip([*proj, conv_cache, cache, slots], [*new, start_conv, start, want_slots]):
            dst.copy_(src)
        unrelated_eager_work(t)
        graph.replay()
        t.cuda.synchronize()
        assert all(same(a, c) for a, c in zip(outs, want)), replay
        assert same(cache, eager) and same(conv_cache, eager_conv), replay


def test_graph_of_gradients():
    """conv and norm with their gradients captured, replayed on new inputs, against eager calls."""
    announce("graph of gradients")
    t = torch()
    r = Rand(740)
    b, d, L = 2, 136, 333
    mk = lambda s: r(s, "bf16")[0]
    x, z, g = mk((b, L, d)), mk((b, L, d)), mk((b, L, d))
    w, bias, nw = r((d, 4))[0], r((d,))[0], r((d,))[0]

    def work():
        xt, zt = x.transpose(1, 2), z.transpose(1, 2)
        u, fin = ssm.conv(xt, w, bias=bias, silu=True)
        out, rstd = ssm.norm_train(u, nw, z=zt, token_major=True)
        gn = ssm.norm_backward(u, nw, rstd, g, z=zt, token_major=True)
        gc = ssm.conv_backward(xt, w, gn["dy"], bias=bias, silu=True)
        return [u, fin, out, rstd, *gn.values(), gc["dx"], gc["dweight"], gc["dbias"]]

    graph, got = capture(t, work)
    for replay in range(3):
        for buf in (x, z, g):
            buf.copy_(mk((b, L, d)))
        unrelated_eager_work(t)
        graph.replay()
        t.cuda.synchronize()
        got_now = [v.clone() for v in got]
        for a, c in zip(got_now, work()):
            assert same(a.contiguous(), c.contiguous()), replay


def test_two_streams_at_once():
    """Independent calls on two streams, each waiting for inputs made on its own."""
    announce("two streams")
    t = torch()
    w, nw = t.randn(512, 4, device="cuda"), t.randn(512, device="cuda")
    results = {}
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    t.cuda.synchronize()
    for k in range(6):
        for i, s in enumerate(streams):
            with t.cuda.stream(s):
                x = t.randn(2, 512, 700, device="cuda", generator=t.Generator("cuda").manual_seed(i))
                u, _ = ssm.conv(x, w, silu=True)
                y, rstd = ssm.norm_train(u, nw)
                gr = ssm.norm_backward(u, nw, rstd, x)
                gc = ssm.conv_backward(x, w, gr["dy"], silu=True)
                results[(k, i)] = [u, y, gr["dy"], gr["dweight"], gc["dx"], gc["dweight"]]
    t.cuda.synchronize()
    for i in range(2):
        for k in range(1, 6):
            assert all(same(a, c) for a, c in zip(results[(0, i)], results[(k, i)])), (k, i)
    assert not same(results[(0, 0)][0], results[(0, 1)][0])


# ---------------------------------------------------------------- the binding

def test_both_ways_of_marshalling_agree(monkeypatch):
    """The extension module's way and the checks in Python (which it leaves calls to by returning
    None) make the same calls."""
    announce("both ways of marshalling")
    t = torch()
    from selective_state_space_fwd_amd import block

    class Never:
        conv = conv_step = state_step = norm = staticmethod(lambda *a: None)
        conv_backward = norm_backward = staticmethod(lambda *a: None)

    r = Rand(750)
    x, w, bias = r((2, 40, 50), "bf16")[0], r((40, 4))[0], r((40,))[0]
    init, lengths = r((2, 40, 3), "bf16")[0], t.tensor([50, 7], dtype=t.int32, device="cuda")
    row, tok = r((3, 40), "bf16")[0], x.transpose(1, 2).contiguous().transpose(1, 2)
    A1, A2, D_, B = -r((40, 8))[0].abs(), -r((4,))[0].abs(), r((40,))[0], r((3, 8), "bf16")[0]
    slots = t.tensor([2, 0, 1], dtype=t.int32, device="cuda")
    dt4, b4 = r((3, 4), "bf16")[0], r((4,))[0]

    def calls():
        cs, st = t.zeros(3, 40, 3, device="cuda", dtype=t.bfloat16), t.ones(3, 40, 8, device="cuda")
        got = [*ssm.conv(x, w, bias=bias, silu=True, initial_state=init, lengths=lengths),
               ssm.conv(tok, w, return_final_state=False)[0],
               ssm.conv_step(row, cs, w, bias, True, slots), cs,
               ssm.scan_step(row, row, A1, B, B, st, D=D_, z=row, delta_bias=bias,
                             delta_softplus=True, slots=slots),
               ssm.ssd_step(row, dt4, A2, B, B, st, D=D_, dt_bias=b4, dt_softplus=True), st,
               ssm.norm(tok, bias, z=x, eps=1e-3, groups=5, token_major=True),
               *ssm.norm_train(x, bias, norm_before_gate=True, z=x)]
        for g in (ssm.conv_backward(tok, w, x, bias=bias, silu=True, initial_state=init,
                                    lengths=lengths, dfinal=init),
                  ssm.conv_backward(x, w, x, want_dinitial=True),
                  ssm.norm_backward(tok, bias, got[-1], x, z=x),
                  ssm.norm_backward(x, bias, got[-1], tok.transpose(1, 2), token_major=True)):
            got += [v for v in g.values() if v is not None]
        return got

    native = calls()
    assert all(v is not None for v in (block._binding.conv(x, w, None, False, None, None, None, None, True),
                                       block._binding.norm(x, bias, None, 1e-5, 1, False, False, None, False),
                                       block._binding.conv_backward(tok, w, x, None, False, None, None, None,
                                                                    None, None)))
    monkeypatch.setattr(block, "_binding", Never)
    for a, c in zip(native, calls()):
        assert a.shape == c.shape and a.stride() == c.stride() and same(a.contiguous(), c.contiguous())


@pytest.mark.parametrize("L", [1, 5])
@pytest.mark.parametrize("d", [1, 6])
def test_norm_of_views_contiguous_both_ways(d, L):
    """One channel, one step, and overlapping views whose steps and channels are both one element
    apart: every such y and z, both results' orders, gradients included."""
    announce(f"norm views contiguous both ways d{d} L{L}")
    t = torch()
    r = Rand(770 + 10 * d + L)
    b = 2
    kinds = []
    for _ in range(2):
        v = r((b, d, L))
        token = v[0].transpose(1, 2).contiguous().transpose(1, 2)
        flat = r((b * (d + L),))[0]
        both = flat.as_strided((b, d, L), (d + L - 1, 1, 1))
        kinds.append([v[0], token, both])
    w, w64 = r((d,))
    dout, dout64 = r((b, d, L))
    for y in kinds[0]:
        for z in [None] + kinds[1]:
            for token in (False, True):
                z64 = None if z is None else host(z)
                out, rstd = ssm.norm_train(y, w, z=z, token_major=token)
                ref, rref = ob.norm_ref(host(y), w64, z64, 1e-5, 1)
                check(out, ref.transpose(0, 2, 1) if token else ref, TOL["f32"], "out")
                g = ssm.norm_backward(y, w, rstd, dout.transpose(1, 2) if token else dout, z=z,
                                      token_major=token)
                c = ssm.norm_backward(y.contiguous(), w, rstd, dout,
                                      z=None if z is None else z.contiguous())
                for k in g:
                    assert g[k] is c[k] is None or same(g[k].contiguous(), c[k].contiguous()), k


@pytest.mark.parametrize("L", [1, 9])
def test_gradients_of_sums(L):
    """The gradient that a sum hands back is one element read everywhere (strides of zero)."""
    announce(f"gradients of sums L{L}")
    t = torch()
    r = Rand(780 + L)
    v = {k: r(s) for k, s in
         (("y", (2, 20, L)), ("w", (20, 4)), ("weight", (20,)), ("z", (2, 20, L)))}
    x, w, nw, z = (v[k][0].requires_grad_() for k in ("y", "w", "weight", "z"))
    ones = np.ones((2, 20, L))
    v["dout"] = (None, ones)
    tol = grad_tol("f32", v, (2, 20, L, 1), "gate_first")
    ref = ob.norm_bwd_ref(v["y"][1], v["weight"][1], ones, v["z"][1], 1e-5)
    for token in (False, True):
        out = ssm.gated_norm(x, nw, z=z, token_major=token)
        dy, dweight, dz = t.autograd.grad(out.sum(), [x, nw, z])
        check(dy, ref["dy"], tol, "dy")
        check(dz, ref["dz"], tol, "dz")
        check(dweight, ref["dweight"], sum_tol(2 * L), "norm dweight")
    ref = ob.conv_bwd_ref(v["y"][1], v["w"][1], ones, silu=True, dfinal=np.ones((2, 20, 3)))
    out, fin = ssm.causal_conv(x, w, silu=True)
    dx, dw = t.autograd.grad(out.sum() + fin.sum(), [x, w])
    check(dx, ref["dx"], TOL["f32"], "dx")
    check(dw, ref["dweight"], sum_tol(2 * L), "conv dweight")


@pytest.mark.parametrize("order", ["time", "channel"])
def test_tensors_past_32_bits(order):
    """More than 2^31 elements: the last batch row of the convolution and of the norm, both
    directions, as a call of that row alone gives it, bit for bit."""
    announce(f"tensors past 32 bits {order}")
    t = torch()
    d, L = 1031, 1050001
    assert 2 * d * L > 1 << 31
    g = t.Generator("cuda").manual_seed(790)
    shape = (2, d, L) if order == "time" else (2, L, d)
    draw = lambda: t.randn(shape, device="cuda", dtype=t.bfloat16, generator=g)
    view = (lambda v: v) if order == "time" else (lambda v: v.transpose(1, 2))
    x = view(draw())
    w, nw = t.randn(d, 4, device="cuda", generator=g), t.randn(d, device="cuda", generator=g)
    lengths = t.tensor([5, L - 3], dtype=t.int32, device="cuda")

    def equal(a, c, label):
        assert a.stride()[1:] == c.stride()[1:]
        dense = lambda v: v if v.is_contiguous() else v.transpose(1, 2)
        assert t.equal(dense(a[1:]).view(t.int16 if a.dtype == t.bfloat16 else t.int32),
                       dense(c).view(t.int16 if a.dtype == t.bfloat16 else t.int32)), label

    out, fin = ssm.conv(x, w, silu=True, lengths=lengths)
    out1, fin1 = ssm.conv(x[1:], w, silu=True, lengths=lengths[1:])
    equal(out, out1, "conv")
    equal(fin, fin1, "final state")
    assert not out[0, :, 5:].any()
    dx = ssm.conv_backward(x, w, out, silu=True, lengths=lengths)["dx"]
    equal(dx, ssm.conv_backward(x[1:], w, out1, silu=True, lengths=lengths[1:])["dx"], "conv dx")
    del out, out1, dx
    out, rstd = ssm.norm_train(x, nw, z=x, token_major=order == "channel")
    out1, rstd1 = ssm.norm_train(x[1:], nw, z=x[1:], token_major=order == "channel")
    equal(out, out1, "norm")
    equal(rstd, rstd1, "rstd")
    gr = ssm.norm_backward(x, nw, rstd, out, z=x, token_major=order == "channel")
    gr1 = ssm.norm_backward(x[1:], nw, rstd1, out1, z=x[1:], token_major=order == "channel")
    equal(gr["dy"], gr1["dy"], "norm dy")
    equal(gr["dz"], gr1["dz"], "norm dz")
    assert bool(t.isfinite(gr["dweight"]).all())


def test_outputs_given_and_arguments_copied():
    """Outputs passed in are returned; strided weights, states and lengths are copied."""
    announce("outputs given")
    t = torch()
    r = Rand(760)
    x, x64 = r((2, 12, 30))
    w2, w264 = r((12, 8))
    out, fin = t.empty(2, 12, 30, device="cuda"), t.empty(2, 12, 3, device="cuda")
    got = ssm.conv(x, w2[:, ::2], out=out, final_state=fin)
    assert got[0] is out and got[1] is fin
    check(out, ob.conv_ref(x64, w264[:, ::2])[0], TOL["f32"], "strided weight")
    st = t.zeros(2, 12, 3, device="cuda")
    o = t.empty(2, 12, device="cuda")
    rows = x[:, :, 3]                                     # last axis strided: copied
    assert ssm.conv_step(rows, st, w2[:, :4].contiguous(), out=o) is o
    check(o, x64[:, :, 3] * w264[:, 3], TOL["f32"], "strided row")
    y = t.empty(2, 30, 12, device="cuda")
    assert ssm.norm(x, w2[:, 0], token_major=True, out=y) is y
    check(y, ob.norm_ref(x64, w264[:, 0])[0].transpose(0, 2, 1), TOL["f32"], "norm")
    ws = t.empty(ssm.ssm_conv_bwd_workspace_bytes(2, 12, 4, 30, ssm.SSM_IO_F32), device="cuda",
                 dtype=t.uint8)
    a = ssm.conv_backward(x, w2[:, :4].contiguous(), out, workspace=ws)
    c = ssm.conv_backward(x, w2[:, :4].contiguous(), out)
    assert same(a["dx"], c["dx"]) and same(a["dweight"], c["dweight"])


def test_refusals():
    announce("refusals")
    t = torch()
    f = lambda *s: t.zeros(*s, device="cuda")
    h = lambda *s: t.zeros(*s, device="cuda", dtype=t.bfloat16)
    i32 = t.zeros(2, dtype=t.int32, device="cuda")
    x, w = f(2, 8, 16), f(8, 4)
    types = [
        lambda: ssm.conv(x.half(), w), lambda: ssm.conv(x, w.bfloat16()),
        lambda: ssm.conv(x, w, bias=h(8)), lambda: ssm.conv(x, w, initial_state=h(2, 8, 3)),
        lambda: ssm.conv(x, w, lengths=i32.long()), lambda: ssm.conv(x, w, out=h(2, 8, 16)),
        lambda: ssm.conv_backward(x, w, h(2, 8, 16)),
        lambda: ssm.conv_step(x[:, :, 0].contiguous(), h(2, 8, 3), w),
        lambda: ssm.conv_step(f(2, 8), f(2, 8, 3), w, slots=i32.long()),
        lambda: ssm.scan_step(f(2, 8), h(2, 8), f(8, 4), f(2, 4), f(2, 4), f(2, 8, 4)),
        lambda: ssm.scan_step(h(2, 8), h(2, 8), f(8, 4), h(2, 4), h(2, 4), h(2, 8, 4)),
        lambda: ssm.norm(x, h(8)), lambda: ssm.norm(x, f(8), z=h(2, 8, 16)),
        lambda: ssm.norm_backward(x, f(8), h(2, 1, 16), x),
    ]
    values = [
        lambda: ssm.conv(x, f(7, 4)), lambda: ssm.conv(x[0], w), lambda: ssm.conv(x, w, bias=f(7)),
        lambda: ssm.conv(x, w, initial_state=f(2, 8, 4)), lambda: ssm.conv(x, w, lengths=i32[:1]),
        lambda: ssm.conv(x, w.cpu()), lambda: ssm.conv(x, w, out=f(2, 16, 8).transpose(1, 2)),
        lambda: ssm.conv_backward(x, w, f(2, 8, 15)),
        lambda: ssm.conv_backward(x, w, x, workspace=f(4)),
        lambda: ssm.conv_step(f(2, 8), f(2, 7, 3), w), lambda: ssm.conv_step(f(2, 8), f(2, 8, 2), w),
        lambda: ssm.conv_step(f(2, 8), f(2, 3, 8).transpose(1, 2), w),
        lambda: ssm.scan_step(f(2, 8), f(2, 8), f(8, 4), f(2, 5), f(2, 4), f(2, 8, 4)),
        lambda: ssm.scan_step(f(2, 8), f(2, 8), f(8, 4), f(2, 4), f(2, 4), f(2, 4, 8).transpose(1, 2)),
        lambda: ssm.ssd_step(f(2, 8), f(2, 8), f(4), f(2, 4), f(2, 4), f(2, 8, 4)),
        lambda: ssm.ssd_step(f(2, 8), f(2, 3), f(3), f(2, 4), f(2, 4), f(2, 8, 4)),
        lambda: ssm.norm(x, f(7)), lambda: ssm.norm(x, f(8), groups=3), lambda: ssm.norm(x, f(8), groups=0),
        lambda: ssm.norm(x, f(8), z=f(2, 8, 15)), lambda: ssm.norm(x, f(8), z=x.cpu()),
        lambda: ssm.norm(x, f(8), token_major=True, out=f(2, 8, 16)),
        lambda: ssm.norm_backward(x, f(8), f(2, 1, 15), x),
        lambda: ssm.norm_backward(x, f(8), f(2, 1, 16), x, token_major=True),
    ]
    refused = [  # by the C ABI
        lambda: ssm.conv(x, f(8, 5)), lambda: ssm.conv(x, f(8, 1)),
        lambda: ssm.conv(x, w, out=x), lambda: ssm.norm(x, f(8), out=x),
        lambda: ssm.norm(x, f(8), eps=-1.0), lambda: ssm.norm(x, f(8), eps=float("nan")),
        lambda: ssm.conv_step(f(2, 8), f(1, 8, 3), w),     # fewer slots than rows
        lambda: ssm.scan_step(f(2, 8), f(2, 8), f(8, 300), f(2, 300), f(2, 300), f(2, 8, 300)),
        lambda: ssm.conv_backward(x, w, x, workspace=t.empty(1, dtype=t.uint8, device="cuda")),
    ]
    for group, error in ((types, TypeError), (values, ValueError), (refused, ssm.SsmScanError)):
        for k, call in enumerate(group):
            with pytest.raises(error):
                call()
                print("not refused:", error, k)
    state = f(2, 8, 4)
    with pytest.raises(ssm.SsmScanError):  # out inside the state
        ssm.scan_step(f(2, 8), f(2, 8), f(8, 4), f(2, 4), f(2, 4), state, out=state.view(-1)[:16].view(2, 8))
    t.cuda.synchronize()
