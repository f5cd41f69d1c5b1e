"""Linear attention and the queries' and keys' norm as a layer uses them: a prompt, its state in a
cache and tokens from it; training through autograd; captured and replayed graphs; two streams;
both ways of marshalling a call; refusals on the device."""
import numpy as np
import pytest

import selective_state_space_fwd_amd as ssm
from block_util import Rand, same
from gpu_util import announce, host, torch
from linattn_util import Attention, within
from oracle import linattn as ol
from selective_state_space_fwd_amd import block
from test_gpu_block import capture
from test_gpu_graph import unrelated_eager_work

pytestmark = pytest.mark.gpu

HK, H, DK, DV, PAIRS = 2, 4, 64, 32, 16
WIDE = 2 * HK * DK + 2 * H * DV


class Layer:
    """Between a layer's projections: queries, keys, values and the gate cut from one projection, the
    norm and rotation, the attention, and the gated norm of its result."""

    def __init__(self, seed, places=256):
        t, r = torch(), Rand(seed)
        self.qw, self.kw = r((DK,))[0], r((DK,))[0]
        self.nw = r((H * DV,))[0]
        angle = t.arange(places)[:, None] * 0.3 ** t.arange(PAIRS)
        self.cos, self.sin = angle.cos().cuda(), angle.sin().cuda()

    def cut(self, proj):
        at, parts = 0, []
        for h, d in ((HK, DK), (HK, DK), (H, DV), (H, DV)):
            parts.append(proj[..., at:at + h * d].unflatten(-1, (h, d)))
            at += h * d
        return parts

    def prompt(self, proj, g, lengths=None, positions=None):
        q, k, v, z = self.cut(proj)
        q, k = ssm.qk_norm(q, k, self.qw, self.kw, self.cos, self.sin, positions=positions)
        out, state = ssm.linattn(q, k, v, g, lengths=lengths)
        y = ssm.norm(out.flatten(2).transpose(1, 2), self.nw, z=z.flatten(2).transpose(1, 2),
                     groups=H, token_major=True)
        return y, state

    def token(self, proj, g, cache, slots, positions):
        q, k, v, z = (x[:, None] for x in self.cut(proj))
        q, k = ssm.qk_norm(q, k, self.qw, self.kw, self.cos, self.sin, positions=positions[:, None])
        out = ssm.linattn_step(q[:, 0], k[:, 0], v[:, 0], cache, g, slots=slots)
        return ssm.norm(out.flatten(1)[..., None], self.nw, z=z.flatten(1)[..., None], groups=H,
                        token_major=True)[:, 0]


def test_prompt_then_tokens():
    """A padded batch of prompts, then tokens from their states, is the whole prompt."""
    t = torch()
    announce("layer: prompt then tokens")
    m, r = Layer(800), Rand(801)
    b, L, more = 3, 60, 12
    proj, g = r((b, L + more, WIDE))[0], -r((b, L + more, H))[0].abs()
    lengths = t.tensor([60, 17, 0], dtype=t.int32, device="cuda")
    whole = []
    for i in range(b):  # each request alone: its prompt and its tokens after it
        n = int(lengths[i])
        x = t.cat((proj[i:i + 1, :n], proj[i:i + 1, L:]), 1)
        gi = t.cat((g[i:i + 1, :n], g[i:i + 1, L:]), 1)
        whole.append(m.prompt(x, gi)[0][0])
    y, state = m.prompt(proj[:, :L], g[:, :L], lengths)
    cache, slots = t.full((5, H, DV, DK), float("nan"), device="cuda"), t.tensor([4, 0, 2], dtype=t.int32, device="cuda")
    cache[slots.long()] = state
    got = [m.token(proj[:, L + i], g[:, L + i], cache, slots, lengths + i) for i in range(more)]
    # float32 throughout, the same sums in other orders: a few hundred roundings of values whose scale
    # the norm sets to the weight's, and its own conditioning, under 1e-4 of the results' 2-norm
    for i in range(b):
        n = int(lengths[i])
        a = t.cat((y[i, :n], t.stack([v[i] for v in got])))
        assert (a - whole[i]).norm() <= 1e-4 * whole[i].norm(), i
    assert cache[[1, 3]].isnan().all()


def test_training_layer():
    """Gradients of a layer through autograd against float64 autograd of the same formulas."""
    t = torch()
    announce("layer: training")
    m, r = Layer(810), Rand(811)
    b, L = 2, 90
    proj, proj64 = r((b, L, WIDE))
    g = -r((b, L, H))[0].abs() * 0.2
    s0 = r((b, H, DV, DK))[0]
    dy, ds = r((b, L, H * DV))[0], r((b, H, DV, DK))[0]
    leaves = [x.clone().requires_grad_() for x in (proj, g, s0, m.qw, m.kw, m.nw)]

    def layer(proj, g, s0, qw, kw, nw):
        q, k, v, z = m.cut(proj)
        q, k = ssm.rotary_qk_norm(q, k, qw, kw, m.cos, m.sin)
        out, state = ssm.linear_attention(q, k, v, g, initial_state=s0)
        y = ssm.gated_norm(out.flatten(2).transpose(1, 2), nw, z=z.flatten(2).transpose(1, 2), groups=H,
                           token_major=True)
        return (y * dy).sum() + (state * ds).sum()

    got = t.autograd.grad(layer(*leaves), leaves)

    def plain(proj, g, s0, qw, kw, nw):
        q, k, v, z = m.cut(proj)
        cos, sin = m.cos[:L, None].double().cpu(), m.sin[:L, None].double().cpu()

        def one(x, w):
            y = x * t.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w
            a, c = y[..., :PAIRS], y[..., PAIRS:2 * PAIRS]
            return t.cat((a * cos - c * sin, c * cos + a * sin, y[..., 2 * PAIRS:]), -1)

        q, k = one(q, qw).repeat_interleave(2, 2), one(k, kw).repeat_interleave(2, 2)
        S, outs = s0, []
        for i in range(L):
            S = S * g[:, i].exp()[..., None, None] + v[:, i, :, :, None] * k[:, i, :, None]
            outs.append((S * q[:, i, :, None]).sum(3) * DK ** -0.5)
        out = t.stack(outs, 1)
        x = out * z * t.sigmoid(z)
        y = (x * t.rsqrt((x * x).mean(-1, keepdim=True) + 1e-5)).flatten(2) * nw
        return (y * dy.double().cpu()).sum() + (S * ds.double().cpu()).sum()

    ref = [x.detach().double().cpu().requires_grad_() for x in leaves]
    want = t.autograd.grad(plain(*ref), ref)
    # float32 sums of a few hundred terms through four operators: 1e-4 of each gradient's 2-norm
    for name, x, w in zip(("proj", "g", "s0", "qw", "kw", "nw"), got, want):
        x = x.double().cpu()
        assert (x - w).norm() <= 1e-4 * w.norm(), (name, float((x - w).norm() / w.norm()))


def test_autograd_forms():
    """Gradients only of what asks for them; one decay a head; no decay; unused results."""
    t = torch()
    announce("linear_attention autograd forms")
    a = Attention(2, 50, 1, 3, 24, 20, "f32", "head", [50, 9], True, seed=820)
    q, k, v = (x.nan_to_num(0.0).detach().requires_grad_() for x in (a.q, a.k, a.v))
    g = a.g.clone().requires_grad_()
    out, fin = ssm.linear_attention(q, k, v, g, scale=0.3, initial_state=a.s0, lengths=a.n)
    got = t.autograd.grad((fin * a.ds).sum(), (q, k, v, g), allow_unused=True)
    ref = ol.linattn_bwd_ref(a.q64, a.k64, a.v64, 0 * a.dout64, a.g64, 0.3, a.s064, a.lengths, a.ds64)
    ab = ol.linattn_bwd_ref(*map(np.abs, (a.q64, a.k64, a.v64, 0 * a.dout64)), a.g64, 0.3, np.abs(a.s064),
                            a.lengths, np.abs(a.ds64))
    assert (got[0] == 0).all()
    for x, n in ((got[1], "dk"), (got[2], "dv")):
        within(x, ref[n], ab[n], "f32", a.roundings, n)
    within(got[3], ref["dg"].sum((0, 1)), ab["dg"].sum((0, 1)) * 64, "f32", a.roundings, "dg")
    out, fin = ssm.linear_attention(q, k.detach(), v.detach())
    assert not fin.requires_grad or fin.grad_fn is not None
    out.sum().backward()
    assert q.grad is not None and k.grad is None
    with pytest.raises(RuntimeError):  # no second derivatives
        x, = t.autograd.grad(ssm.linear_attention(q, k, v)[0].square().sum(), q, create_graph=True)
        x.sum().backward()
    cos = t.ones(50, 12, device="cuda", requires_grad=True)
    with pytest.raises(ValueError, match="cos has no gradient"):
        ssm.rotary_qk_norm(q, k, cos=cos, sin=cos)


def test_graph_of_tokens():
    """Tokens of a layer captured once, with a padding row of no slot and no position; replayed."""
    t = torch()
    announce("layer: graph of tokens")
    m, r = Layer(830), Rand(831)
    b, steps = 4, 3
    proj = [r((b, WIDE), "bf16")[0] for _ in range(steps)]
    g = [-r((b, H))[0].abs() for _ in range(steps)]
    slots, pos = (t.zeros(b, dtype=t.int32, device="cuda") for _ in range(2))
    cache = r((6, H, DV, DK))[0]
    graph, outs = capture(t, lambda: [m.token(p, x, cache, slots, pos) for p, x in zip(proj, g)])
    for replay, s in enumerate(([0, 1, 2, -1], [5, 3, 0, 1], [2, -1, -1, 4], [1, 1, 3, 3])):
        new = [r((b, WIDE), "bf16")[0] for _ in range(steps)]
        start = r(tuple(cache.shape))[0]
        want_slots = t.tensor(s, dtype=t.int32, device="cuda")
        want_pos = t.tensor([3, 200, -1, 7], dtype=t.int32, device="cuda") + replay
        eager = start.clone()
        want = [m.token(p, x, eager, want_slots, want_pos) for p, x in zip(new, g)]
        for dst, src in zip([*proj, cache, slots, pos], [*new, start, want_slots, want_pos]):
            dst.copy_(src)
        unrelated_eager_work(t)
        graph.replay()
        t.cuda.synchronize()
        assert all(same(x, y) for x, y in zip(outs, want)) and same(cache, eager), replay


@pytest.mark.parametrize("decay,L", [("token", 200), ("head", 700)])
def test_graph_of_gradients(decay, L):
    """Both operators and their gradients captured (segments and the joined states among them), replayed
    on new inputs, next to a second captured graph with workspaces of its own."""
    t = torch()
    announce(f"graph of gradients {decay} {L}")
    a = Attention(1, L, 2, 4, 64, 64, "bf16", decay, None, True, seed=840)
    w = Rand(841)((64,))[0]
    cos, sin = t.rand(2, L, 32, device="cuda").unbind()

    def work():
        q, k = ssm.qk_norm(a.q, a.k, w, w, cos, sin)
        out, fin = ssm.linattn(q, k, a.v, **a.args())
        d = ssm.linattn_backward(q, k, a.v, out, dfinal=fin, **a.args())
        n = ssm.qk_norm_backward(a.q, a.k, d["dq"], d["dk"], w, w, cos, sin)
        return [q, k, out, fin, *d.values(), *n.values()]

    (graph, got), (second, got2) = capture(t, work), capture(t, work)
    for replay in range(3):
        fresh = Attention(1, L, 2, 4, 64, 64, "bf16", decay, None, True, seed=842 + replay)
        for name in ("q", "k", "v", "g", "s0"):
            getattr(a, name).copy_(getattr(fresh, name))
        want = [x.clone() for x in work()]
        unrelated_eager_work(t)
        graph.replay()
        second.replay()
        t.cuda.synchronize()
        assert all(same(x, y) and same(z, y) for x, y, z in zip(got, want, got2)), replay


def test_two_streams():
    t = torch()
    announce("linattn on two streams")
    sets = [Attention(2, 500, 2, 4, 64, 64, "bf16", "token", None, True, seed=850 + i) for i in range(2)]
    call = lambda a: [*ssm.linattn(a.q, a.k, a.v, **a.args()),
                      *ssm.linattn_backward(a.q, a.k, a.v, a.dout, dfinal=a.ds, **a.args()).values()]
    want = [call(a) for a in sets]
    t.cuda.synchronize()
    streams = [t.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, (s, a) in enumerate(zip(streams, sets)):
            with t.cuda.stream(s):
                got[i].append(call(a))
    t.cuda.synchronize()
    for i in range(2):
        for r in got[i]:
            assert all(same(x, y) for x, y in zip(r, want[i]))


# ---------------------------------------------------------------- the binding

def every_call(seed=860):
    """(the tensors written in place, the call)."""
    t = torch()
    a = Attention(2, 40, 1, 2, 32, 16, "f32", "token", None, True, seed=seed)
    h = Attention(2, 40, 1, 2, 32, 16, "f32", "head", None, True, seed=seed)
    r = Rand(seed + 1)  # (the same for every call of this function)
    cos, sin, w, cache = r((40, 8))[0], r((40, 8))[0], r((32,))[0], a.s0.clone()
    out, fin, o1 = t.empty_like(a.dout), t.empty_like(a.s0), t.empty(2, 2, 16, device="cuda")
    qo, ko = t.empty(2, 40, 1, 32, device="cuda"), t.empty(2, 40, 1, 32, device="cuda")
    ws = t.empty(1 << 24, dtype=t.uint8, device="cuda")
    return [
        ([], lambda: ssm.linattn(a.q, a.k, a.v, a.g, initial_state=a.s0)),
        ([out, fin], lambda: ssm.linattn(h.q, h.k, h.v, h.g, 0.5, out=out, final_state=fin, workspace=ws)),
        ([], lambda: (ssm.linattn(a.q, a.k, a.v, return_final_state=False)[0],)),
        ([], lambda: list(ssm.linattn_backward(a.q, a.k, a.v, a.dout, a.g, initial_state=a.s0, dfinal=a.ds).values())),
        ([], lambda: [x for x in ssm.linattn_backward(h.q, h.k, h.v, h.dout, h.g, want_dinitial=True, workspace=ws).values()]),
        ([], lambda: [x for x in ssm.linattn_backward(a.q, a.k, a.v, a.dout, a.g, want_dg=False).values() if x is not None]),
        ([cache, o1], lambda: (ssm.linattn_step(a.q[:, 0], a.k[:, 0], a.v[:, 0], cache, a.g[:, 0], out=o1), cache)),
        ([qo, ko], lambda: ssm.qk_norm(a.q, a.k, w, None, cos, sin, interleaved=True, q_out=qo, k_out=ko)),
        ([], lambda: ssm.qk_norm(a.q, a.k)),
        ([], lambda: [x for x in ssm.qk_norm_backward(a.q, a.k, a.q, a.k, None, w, cos, sin).values() if x is not None]),
    ]


def test_both_ways_of_marshalling(monkeypatch):
    announce("linattn marshalled both ways")
    with_it = [[x.clone() for x in call()] for _, call in every_call()]
    monkeypatch.setattr(block, "_binding", block._NoModule)
    without = [[x.clone() for x in call()] for _, call in every_call()]
    for x, y in zip(with_it, without):
        assert len(x) == len(y) and all(same(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("native", [True, False])
def test_writes_are_seen_by_autograd(native, monkeypatch):
    t = torch()
    announce(f"linattn writes seen by autograd, module {native}")
    block._load()
    if not native:
        monkeypatch.setattr(block, "_binding", block._NoModule)
    for written, call in every_call():
        for v in written:
            scale = t.ones_like(v, requires_grad=True)
            loss = (v * scale).sum()
            call()
            with pytest.raises(RuntimeError, match="inplace operation"):
                loss.backward()


def test_negative_views():
    """Inputs that are the imaginary part of a conjugate are read as their values."""
    t = torch()
    announce("linattn negative views")
    neg = lambda x: t.complex(t.zeros_like(x), -x).conj().imag
    a = Attention(1, 30, 1, 2, 16, 16, "f32", "token", None, True, seed=870)
    q, k, v, g, s0 = (neg(x.contiguous()) for x in (a.q, a.k, a.v, a.g, a.s0))
    assert q.is_neg()
    got = ssm.linattn(q, k, v, g, initial_state=s0)
    assert all(same(x, y) for x, y in zip(got, ssm.linattn(a.q, a.k, a.v, a.g, initial_state=a.s0)))
    w = t.rand(16, device="cuda")
    got = ssm.qk_norm(q, k, neg(w), w)
    assert all(same(x, y) for x, y in zip(got, ssm.qk_norm(a.q, a.k, w, w)))
    with pytest.raises(ValueError, match="contiguous"):
        ssm.linattn_step(a.q[:, 0], a.k[:, 0], a.v[:, 0], s0)


def test_refusals_on_the_device():
    t = torch()
    announce("linattn refusals")
    a = Attention(2, 10, 2, 4, 16, 8, "f32", "token", None, True, seed=880)
    q, k, v, g, s0 = a.q, a.k, a.v, a.g, a.s0
    bad = [
        (ValueError, lambda: ssm.linattn(q, k[:, :9], v)), (ValueError, lambda: ssm.linattn(q, k, v[:1])),
        (ValueError, lambda: ssm.linattn(q, k, v[:, :, :3])), (TypeError, lambda: ssm.linattn(q, k.bfloat16(), v)),
        (TypeError, lambda: ssm.linattn(q.half(), k.half(), v.half())), (TypeError, lambda: ssm.linattn(q, k, v, g.double())),
        (ValueError, lambda: ssm.linattn(q, k, v, g[:, :, :3])), (ValueError, lambda: ssm.linattn(q, k, v, g[0])),
        (ValueError, lambda: ssm.linattn(q, k, v, initial_state=s0[:1])), (ValueError, lambda: ssm.linattn(q[0], k[0], v[0])),
        (TypeError, lambda: ssm.linattn(q, k, v, initial_state=s0.bfloat16())),
        (TypeError, lambda: ssm.linattn(q, k, v, lengths=t.zeros(2, dtype=t.int64, device="cuda"))),
        (ValueError, lambda: ssm.linattn(q, k, v.cpu())), (ValueError, lambda: ssm.linattn(q.cpu(), k, v)),
        (ValueError, lambda: ssm.linattn(q, k, v, out=t.empty(2, 10, 4, 9, device="cuda"))),
        (ValueError, lambda: ssm.linattn(q, k, v, final_state=s0.transpose(2, 3).contiguous().transpose(2, 3))),
        (ValueError, lambda: ssm.linattn(q, k, v, workspace=t.empty(8, device="cuda"))),
        (ssm.SsmScanError, lambda: ssm.linattn(q, k, v, initial_state=s0, final_state=s0)),
        (ValueError, lambda: ssm.linattn_backward(q, k, v, v[:, :9])), (ValueError, lambda: ssm.linattn_backward(q, k, v, v, want_dg=True)),
        (ssm.SsmScanError, lambda: ssm.linattn_backward(q, k, v, v, workspace=t.empty(8, dtype=t.uint8, device="cuda"))),
        (ValueError, lambda: ssm.linattn_step(q, k, v, s0)), (ValueError, lambda: ssm.linattn_step(q[:, 0], k[:, 0], v[:, 0], s0[:, :3])),
        (ssm.SsmScanError, lambda: ssm.linattn_step(q[:, 0], k[:, 0], v[:, 0], s0[:1].contiguous())),
        (TypeError, lambda: ssm.linattn_step(q[:, 0], k[:, 0], v[:, 0], s0, slots=t.zeros(2, device="cuda"))),
        (ValueError, lambda: ssm.qk_norm(q, k[..., :8])), (ValueError, lambda: ssm.qk_norm(q, k, q_weight=t.ones(8, device="cuda"))),
        (ValueError, lambda: ssm.qk_norm(q, k, cos=t.ones(10, 4, device="cuda"))),
        (ValueError, lambda: ssm.qk_norm(q, k, cos=t.ones(9, 4, device="cuda"), sin=t.ones(9, 4, device="cuda"))),
        (ValueError, lambda: ssm.qk_norm(q, k, cos=t.ones(10, 9, device="cuda"), sin=t.ones(10, 9, device="cuda"))),
        (TypeError, lambda: ssm.qk_norm(q, k.bfloat16())), (ValueError, lambda: ssm.qk_norm(q[0], k[0])),
    ]
    wide = t.zeros(1, 4, 1, 300, device="cuda")
    bad += [(ssm.SsmScanError, lambda: ssm.linattn(wide, wide, wide)), (ssm.SsmScanError, lambda: ssm.qk_norm(wide, wide))]
    for i, (error, call) in enumerate(bad):
        with pytest.raises(error):
            call()
            print("accepted", i)
