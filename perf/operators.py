"""Cases of the operators around the scan in a Mamba block, for timing and comparison.

The operators: the short causal convolution (a prompt, its gradient, one token against a
cache), the single-token state update of Mamba-1 and Mamba-2 against a cache of request
slots, and the gated RMS norm after the scan (and its gradient).

``run`` computes a case in its plain form, elementary torch operations in 32 bits rounded
once at the end, while ``own`` is false, and calls this package while it is true. ``exact``
computes the same outputs from the definitions in 64 bits.

Shapes: x, y, z [batch, dim, seqlen], "channel" memory order (time contiguous, what the scan
takes) or "token" order (channels contiguous, a slice of a projection's output).
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}
_BYTES = {"bf16": 2, "f32": 4}


def _conv(name, op, b, d, L, W, io, order, lengths, state):
    return {"name": name, "op": op, "batch": b, "dim": d, "seqlen": L, "width": W, "io": io,
            "order": order, "lengths": lengths, "state": state}


def _norm(name, op, b, d, L, groups, io, y_order, z_order, out_order, first):
    return {"name": name, "op": op, "batch": b, "dim": d, "seqlen": L, "groups": groups, "io": io,
            "y_order": y_order, "z_order": z_order, "out_order": out_order, "norm_first": first}


def listed():
    return [
        # The convolution ahead of the Mamba-2 layer (2048 channels and two times 128 states),
        # read from the slice of the projection's output that holds them.
        _conv("conv_prompt", "conv", 4, 2304, 2048, 4, "bf16", "token", False, False),
        # One very long fp32 prompt handed on from an earlier chunk, and on to the next.
        _conv("conv_long_f32", "conv", 1, 1536, 65536, 4, "f32", "channel", False, True),
        # A padded bucket of requests of different lengths, an odd size, three taps.
        _conv("conv_ragged", "conv", 5, 523, 777, 3, "bf16", "channel", True, True),
        # Training: the gradient of conv_prompt.
        _conv("conv_grad", "conv_grad", 4, 2304, 2048, 4, "bf16", "token", False, False),
        # One token of eight requests: latency.
        {"name": "conv_step", "op": "conv_step", "batch": 8, "slots": 8, "dim": 2304, "width": 4,
         "io": "bf16"},
        # One token of many requests, out of a larger cache.
        {"name": "conv_step_batch", "op": "conv_step", "batch": 384, "slots": 512, "dim": 4352,
         "width": 4, "io": "bf16"},
        # The Mamba-2 state of eight requests advanced by a token.
        {"name": "ssd_step", "op": "ssd_step", "batch": 8, "slots": 8, "heads": 32, "headdim": 64,
         "dstate": 128, "io": "bf16", "gate": False},
        # Serving at a large batch: the state is all of the work.
        {"name": "ssd_step_batch", "op": "ssd_step", "batch": 256, "slots": 320, "heads": 64,
         "headdim": 64, "dstate": 128, "io": "bf16", "gate": False},
        # The Mamba-1 state, gated, fp32, an odd number of requests.
        {"name": "scan_step", "op": "scan_step", "batch": 61, "slots": 80, "dim": 2048,
         "dstate": 16, "io": "f32", "gate": True},
        # The norm after a layer's scan: the scan's output, the gate in the projection's output,
        # and the result in the order the output projection reads.
        _norm("norm_layer", "norm", 4, 2048, 2048, 1, "bf16", "channel", "token", "token", False),
        # Its gradient.
        _norm("norm_grad", "norm_grad", 4, 2048, 2048, 1, "bf16", "channel", "token", "token",
              False),
        # One token of eight requests.
        _norm("norm_token", "norm", 8, 2048, 1, 1, "bf16", "channel", "token", "token", False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(["conv", "conv", "conv_grad", "conv_step", "ssd_step", "scan_step", "norm",
                     "norm_grad"])
    io = rng.choice(["bf16", "bf16", "f32"])
    if op in ("conv", "conv_grad"):
        most = 1 << (24 if op == "conv" else 23)
        d = _log(rng, 24, 6000)
        L = _log(rng, 1, min(40000, most // d))
        b = _log(rng, 1, max(1, min(16, most // (d * L))))
        c = _conv("", op, b, d, L, rng.choice([2, 3, 4, 4]), io, rng.choice(["token", "channel"]),
                  rng.random() < 0.4, rng.random() < 0.5)
    elif op == "conv_step":
        b = _log(rng, 1, 384)
        c = {"op": op, "batch": b, "slots": b + rng.randrange(0, 64), "dim": _log(rng, 24, 6000),
             "width": rng.choice([2, 3, 4, 4]), "io": io}
    elif op == "ssd_step":
        n = rng.choice([16, 64, 100, 128, 128, 256])
        p = rng.choice([16, 32, 48, 64, 64, 128])
        h = _log(rng, 1, 96)
        b = _log(rng, 1, max(1, min(256, (1 << 26) // (n * p * h))))
        c = {"op": op, "batch": b, "slots": b + rng.randrange(0, 32), "heads": h, "headdim": p,
             "dstate": n, "io": io, "gate": rng.random() < 0.5}
    elif op == "scan_step":
        n = rng.choice([5, 8, 16, 16, 32, 64])
        d = _log(rng, 24, 6000)
        b = _log(rng, 1, max(1, min(256, (1 << 26) // (n * d))))
        c = {"op": op, "batch": b, "slots": b + rng.randrange(0, 32), "dim": d, "dstate": n,
             "io": io, "gate": rng.random() < 0.5}
    else:
        most = 1 << (24 if op == "norm" else 23)
        groups = rng.choice([1, 1, 1, 2, 4, 8])
        d = groups * _log(rng, max(1, 32 // groups), 6000 // groups)
        L = _log(rng, 1, min(8192, most // d))
        b = _log(rng, 1, max(1, min(64, most // (d * L))))
        order = lambda: rng.choice(["token", "channel"])  # noqa: E731
        c = _norm("", op, b, d, L, groups, io, order(), order(), order(), rng.random() < 0.3)
    c.pop("name", None)
    return c


# ------------------------------------------------------------------ inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _rand(g, *shape):
    return torch.rand(shape, device="cuda", generator=g)


def _signal(g, c, order, scale=1.0):
    """[batch, dim, seqlen] values of c's storage type; in token order a slice of a wider
    token-major buffer, as a projection's output is cut."""
    b, d, L = c["batch"], c["dim"], c["seqlen"]
    if order == "channel":
        return (_randn(g, b, d, L) * scale).to(_DTYPE[c["io"]])
    wide = (_randn(g, b, L, d + 128) * scale).to(_DTYPE[c["io"]])
    return wide[:, :, 64:64 + d].transpose(1, 2)


def _slots(g, c):
    """batch distinct slots of the cache, in no order (None: row i is slot i)."""
    if c["slots"] == c["batch"]:
        return None
    return torch.argsort(_rand(g, c["slots"]))[:c["batch"]].to(torch.int32)


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    op, dt = c["op"], _DTYPE[c["io"]]
    s = {"case": c}
    if op in ("conv", "conv_grad"):
        b, d, L, W = c["batch"], c["dim"], c["seqlen"], c["width"]
        s["x"] = _signal(g, c, c["order"])
        s["weight"] = (_rand(g, d, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (_rand(g, d) * 2 - 1) / math.sqrt(W)
        s["initial"] = _randn(g, b, d, W - 1).to(dt) if c["state"] else None
        s["lengths"] = (_rand(g, b) * (L + 1)).to(torch.int32) if c["lengths"] else None
        if op == "conv_grad":
            s["dout"] = _randn(g, b, d, L).to(dt)
            s["dfinal"] = _randn(g, b, d, W - 1).to(dt) if c["state"] else None
    elif op == "conv_step":
        b, d, W = c["batch"], c["dim"], c["width"]
        s["x"] = _randn(g, b, d + 128).to(dt)[:, 64:64 + d]
        s["state"] = _randn(g, c["slots"], d, W - 1).to(dt)
        s["weight"] = (_rand(g, d, W) * 2 - 1) / math.sqrt(W)
        s["bias"] = (_rand(g, d) * 2 - 1) / math.sqrt(W)
        s["slots"] = _slots(g, c)
    elif op in ("ssd_step", "scan_step"):
        b, n = c["batch"], c["dstate"]
        d = c["heads"] * c["headdim"] if op == "ssd_step" else c["dim"]
        steps = c["heads"] if op == "ssd_step" else d
        if op == "ssd_step":  # x, B and C are parts of the convolution's output row
            row = _randn(g, b, d + 2 * n).to(dt)
            s["x"], s["B"], s["C"] = row[:, :d], row[:, d:d + n], row[:, d + n:]
            s["A"] = -(1 + 15 * _rand(g, steps))
        else:
            s["x"] = _randn(g, b, d).to(dt)
            row = _randn(g, b, 2 * n).to(dt)
            s["B"], s["C"] = row[:, :n], row[:, n:]
            s["A"] = -torch.arange(1, n + 1, device="cuda").float() * (0.5 + _rand(g, d, n))
        s["dt"] = (0.5 * _randn(g, b, steps)).to(dt)
        s["dt_bias"] = torch.log(torch.expm1(1e-3 + 0.099 * _rand(g, steps)))
        s["D"] = _randn(g, d)
        s["z"] = _randn(g, b, d).to(dt) if c["gate"] else None
        s["state"] = _randn(g, c["slots"], d, n)
        s["slots"] = _slots(g, c)
    else:
        s["y"] = _signal(g, c, c["y_order"])
        s["z"] = _signal(g, c, c["z_order"])
        s["weight"] = 1 + 0.1 * _randn(g, c["dim"])
        if op == "norm_grad":
            b, d, L = c["batch"], c["dim"], c["seqlen"]
            token = c["out_order"] == "token"
            s["dout"] = _randn(g, *((b, L, d) if token else (b, d, L))).to(dt)
            v = s["y"].double()
            if not c["norm_first"]:
                zd = s["z"].double()
                v = v * zd / (1 + torch.exp(-zd))
            v = v.reshape(b, c["groups"], d // c["groups"], L)
            s["rstd"] = torch.rsqrt((v * v).mean(2) + 1e-5).float()  # as the forward saved it
    return s


# ------------------------------------------------------------------ plain forms

def _silu(x):
    return x * torch.sigmoid(x)


def _silu_grad(x):
    s = torch.sigmoid(x)
    return s * (1 + x * (1 - s))


def _extended(s, c, to=torch.float32):
    """The window's inputs e: the initial state (zero without one), then x."""
    x = s["x"].to(to)
    first = s["initial"].to(to) if s["initial"] is not None else x.new_zeros(
        (c["batch"], c["dim"], c["width"] - 1))
    return torch.cat((first, x), 2)


def _live(s, c):
    """[batch, 1, seqlen] truth values of the steps before each row's end, or None."""
    if s["lengths"] is None:
        return None
    return (torch.arange(c["seqlen"], device="cuda") < s["lengths"][:, None])[:, None]


def _tail_index(s, c):
    """[batch, 1, width-1] places in e of the last inputs before each row's end."""
    k = torch.arange(c["width"] - 1, device="cuda")
    ends = s["lengths"].long()[:, None] if s["lengths"] is not None else torch.full(
        (c["batch"], 1), c["seqlen"], device="cuda")
    return (ends + k)[:, None]


def _plain_conv(s, c):
    L, W, w = c["seqlen"], c["width"], s["weight"]
    e, live = _extended(s, c), _live(s, c)
    out = _silu(sum(w[:, j, None] * e[:, :, j:j + L] for j in range(W)) + s["bias"][:, None])
    if live is not None:
        out = out * live
    final = torch.gather(e, 2, _tail_index(s, c).expand(-1, c["dim"], -1))
    return out.to(s["x"].dtype), final.to(s["x"].dtype)


def _plain_conv_grad(s, c):
    L, W, w = c["seqlen"], c["width"], s["weight"]
    e, live = _extended(s, c), _live(s, c)
    p = sum(w[:, j, None] * e[:, :, j:j + L] for j in range(W)) + s["bias"][:, None]
    dp = s["dout"].float() * _silu_grad(p)
    if live is not None:
        dp = dp * live
    dw = torch.stack([(dp * e[:, :, j:j + L]).sum((0, 2)) for j in range(W)], 1)
    pad = torch.nn.functional.pad(dp, (W - 1, W - 1))
    de = sum(w[:, j, None] * pad[:, :, W - 1 - j:W - 1 - j + L + W - 1] for j in range(W))
    if s["dfinal"] is not None:
        de.scatter_add_(2, _tail_index(s, c).expand(-1, c["dim"], -1), s["dfinal"].float())
    dt = s["x"].dtype
    grads = {"dx": de[:, :, W - 1:].to(dt), "dweight": dw, "dbias": dp.sum((0, 2))}
    if c["state"]:
        grads["dinitial"] = de[:, :, :W - 1].to(dt)
    return grads


def _rows(s):
    return slice(None) if s["slots"] is None else s["slots"].long()


def _plain_conv_step(s, c):
    at = _rows(s)
    window = torch.cat((s["state"][at], s["x"][:, :, None]), 2)
    out = _silu((window.float() * s["weight"]).sum(2) + s["bias"])
    s["state"][at] = window[:, :, 1:]
    return out.to(s["x"].dtype), s["state"]


def _plain_step(s, c):
    at, x = _rows(s), s["x"].float()
    dt = s["dt"].float() + s["dt_bias"]
    dt = torch.where(dt > 20, dt, torch.log1p(torch.exp(dt)))
    if c["op"] == "ssd_step":
        keep = torch.exp(dt * s["A"]).repeat_interleave(c["headdim"], 1)[:, :, None]
        dt = dt.repeat_interleave(c["headdim"], 1)
    else:
        keep = torch.exp(dt[:, :, None] * s["A"])
    h = s["state"][at] * keep + (dt * x)[:, :, None] * s["B"].float()[:, None]
    y = (h * s["C"].float()[:, None]).sum(2) + s["D"] * x
    if s["z"] is not None:
        y = y * _silu(s["z"].float())
    s["state"][at] = h
    return y.to(s["x"].dtype), s["state"]


def _grouped(t, c):
    return t.float().reshape(c["batch"], c["groups"], c["dim"] // c["groups"], c["seqlen"])


def _in_order(t, order):
    """[batch, dim, seqlen] values as the tensor of the memory order that is asked for."""
    return t.transpose(1, 2).contiguous() if order == "token" else t.contiguous()


def _plain_norm(s, c):
    y, gate = _grouped(s["y"], c), _silu(_grouped(s["z"], c))
    w = s["weight"].reshape(c["groups"], -1, 1)
    v = y if c["norm_first"] else y * gate
    out = v * torch.rsqrt((v * v).mean(2, keepdim=True) + 1e-5) * w
    if c["norm_first"]:
        out = out * gate
    return _in_order(out.reshape(s["y"].shape).to(s["y"].dtype), c["out_order"])


def _plain_norm_grad(s, c):
    y, z, shape = _grouped(s["y"], c), _grouped(s["z"], c), s["y"].shape
    g = _grouped(s["dout"].transpose(1, 2) if c["out_order"] == "token" else s["dout"], c)
    w, r = s["weight"].reshape(c["groups"], -1, 1), s["rstd"][:, :, None]
    gate = _silu(z)
    if c["norm_first"]:
        dz = g * y * r * w * _silu_grad(z)
        g, v = g * gate, y
    else:
        v = y * gate
    dv = r * (w * g - v * (r * r) * (w * g * v).mean(2, keepdim=True))
    dweight = (g * v * r).sum((0, 3)).reshape(-1)
    if c["norm_first"]:
        dy = dv
    else:
        dy, dz = dv * gate, dv * y * _silu_grad(z)
    dt = s["y"].dtype
    return {"dy": dy.reshape(shape).to(dt), "dz": dz.reshape(shape).to(dt), "dweight": dweight}


_PLAIN = {"conv": _plain_conv, "conv_grad": _plain_conv_grad, "conv_step": _plain_conv_step,
          "ssd_step": _plain_step, "scan_step": _plain_step, "norm": _plain_norm,
          "norm_grad": _plain_norm_grad}


def _call(s, c):
    import selective_state_space_fwd_amd as ssm

    op = c["op"]
    if op == "conv":
        return ssm.conv(s["x"], s["weight"], bias=s["bias"], silu=True, initial_state=s["initial"],
                        lengths=s["lengths"])
    if op == "conv_grad":
        grads = ssm.conv_backward(s["x"], s["weight"], s["dout"], bias=s["bias"], silu=True,
                                  initial_state=s["initial"], lengths=s["lengths"],
                                  dfinal=s["dfinal"])
        return {k: grads[k] for k in ("dx", "dweight", "dbias", "dinitial") if grads[k] is not None}
    if op == "conv_step":
        out = ssm.conv_step(s["x"], s["state"], s["weight"], bias=s["bias"], silu=True,
                            slots=s["slots"])
        return out, s["state"]
    if op == "ssd_step":
        out = ssm.ssd_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"],
                           z=s["z"], dt_bias=s["dt_bias"], dt_softplus=True, slots=s["slots"])
        return out, s["state"]
    if op == "scan_step":
        out = ssm.scan_step(s["x"], s["dt"], s["A"], s["B"], s["C"], s["state"], D=s["D"],
                            z=s["z"], delta_bias=s["dt_bias"], delta_softplus=True,
                            slots=s["slots"])
        return out, s["state"]
    token = c["out_order"] == "token"
    if op == "norm":
        return ssm.norm(s["y"], s["weight"], z=s["z"], eps=1e-5, groups=c["groups"],
                        norm_before_gate=c["norm_first"], token_major=token)
    grads = ssm.norm_backward(s["y"], s["weight"], s["rstd"], s["dout"], z=s["z"],
                              groups=c["groups"], norm_before_gate=c["norm_first"],
                              token_major=token)
    return {k: grads[k] for k in ("dy", "dz", "dweight")}


def run(state):
    c = state["case"]
    return _call(state, c) if own else _PLAIN[c["op"]](state, c)


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, op, e = case, case["op"], _BYTES[case["io"]]
    b = c["batch"]
    if op in ("conv", "conv_grad"):
        d, W = c["dim"], c["width"]
        n, edge = b * d * c["seqlen"], b * d * (W - 1)
        params = d * (W + 1) * 4
        if op == "conv":
            return {"bytes": 2 * n * e + edge * e * (2 if c["state"] else 1) + params,
                    "flops": n * (2 * W + 5)}
        return {"bytes": 3 * n * e + edge * e * (3 if c["state"] else 0) + 2 * params,
                "flops": n * (6 * W + 10)}
    if op == "conv_step":
        d, W = c["dim"], c["width"]
        return {"bytes": b * d * e * (2 + 2 * (W - 1)) + d * (W + 1) * 4,
                "flops": b * d * (2 * W + 5)}
    if op in ("ssd_step", "scan_step"):
        d = c["heads"] * c["headdim"] if op == "ssd_step" else c["dim"]
        steps = c["heads"] if op == "ssd_step" else d
        n = c["dstate"]
        rows = b * e * (d * (3 if c["gate"] else 2) + steps + 2 * n)
        params = 4 * (d + steps + (steps if op == "ssd_step" else d * n))
        return {"bytes": b * d * n * 8 + rows + params, "flops": b * d * n * 5 + b * d * 8}
    n = b * c["dim"] * c["seqlen"]
    if op == "norm":
        return {"bytes": 3 * n * e + c["dim"] * 4, "flops": n * 10}
    return {"bytes": 5 * n * e + c["dim"] * 8 + b * c["groups"] * c["seqlen"] * 4, "flops": n * 20}


# ------------------------------------------------------------------ 64 bits, from the definitions

def _exact_conv(s, c):
    """Each output as a product over the window's places, in a strided view of the inputs."""
    e = _extended(s, c, torch.float64)
    w, W = s["weight"].double(), c["width"]
    p = torch.matmul(e.unfold(2, W, 1), w[:, :, None])[..., 0] + s["bias"].double()[:, None]
    return e, w, p


def exact(case, seed):
    c, s = dict(case), prepare(case, seed)
    op = c["op"]
    d64 = lambda t: None if t is None else t.double()  # noqa: E731
    if op in ("conv", "conv_grad"):
        b, L, W = c["batch"], c["seqlen"], c["width"]
        e, w, p = _exact_conv(s, c)
        ends = [L] * b if s["lengths"] is None else s["lengths"].tolist()
        sig = 1 / (1 + torch.exp(-p))
        if op == "conv":
            out = p * sig
            for i, n in enumerate(ends):
                out[i, :, n:] = 0
            final = torch.stack([e[i, :, n:n + W - 1] for i, n in enumerate(ends)])
            return out, final
        dp = d64(s["dout"]) * (sig + p * sig * (1 - sig))
        for i, n in enumerate(ends):
            dp[i, :, n:] = 0
        dw = torch.matmul(dp.transpose(0, 1).reshape(c["dim"], 1, b * L),
                          e.unfold(2, W, 1).transpose(0, 1).reshape(c["dim"], b * L, W))[:, 0]
        de = torch.zeros_like(e)
        for j in range(W):  # the step t reads the places t .. t + W - 1
            de[:, :, j:j + L] += w[:, j, None] * dp
        if s["dfinal"] is not None:
            for i, n in enumerate(ends):
                de[i, :, n:n + W - 1] += d64(s["dfinal"])[i]
        grads = {"dx": de[:, :, W - 1:], "dweight": dw, "dbias": dp.sum((0, 2))}
        if c["state"]:
            grads["dinitial"] = de[:, :, :W - 1]
        return grads
    if op == "conv_step":
        rows = list(range(c["batch"])) if s["slots"] is None else s["slots"].tolist()
        window = torch.cat((d64(s["state"])[rows], d64(s["x"])[:, :, None]), 2)
        p = (window * d64(s["weight"])).sum(2) + d64(s["bias"])
        state = d64(s["state"])
        state[rows] = window[:, :, 1:]
        return p / (1 + torch.exp(-p)), state
    if op in ("ssd_step", "scan_step"):
        rows = list(range(c["batch"])) if s["slots"] is None else s["slots"].tolist()
        n, x = c["dstate"], d64(s["x"])
        step = torch.nn.functional.softplus(d64(s["dt"]) + d64(s["dt_bias"]))
        A = d64(s["A"])
        if op == "ssd_step":  # channel h * headdim + p has head h's step size and A
            head = torch.arange(x.shape[1], device="cuda") // c["headdim"]
            step, A = step[:, head], A[head][:, None].expand(-1, n)
        state = d64(s["state"])
        y = torch.empty_like(x)
        for i, r in enumerate(rows):
            state[r] = torch.exp(step[i][:, None] * A) * state[r] + torch.outer(
                step[i] * x[i], d64(s["B"][i]))
            y[i] = torch.mv(state[r], d64(s["C"][i]))
        y = y + d64(s["D"]) * x
        if s["z"] is not None:
            z = d64(s["z"])
            y = y * (z / (1 + torch.exp(-z)))
        return y, state
    b, d, L, k = c["batch"], c["dim"], c["seqlen"], c["groups"]
    tokens = lambda t: d64(t).transpose(1, 2).reshape(b, L, k, d // k)  # noqa: E731
    y, z, w = tokens(s["y"]), tokens(s["z"]), d64(s["weight"]).reshape(k, d // k)
    sig = 1 / (1 + torch.exp(-z))
    v = y if c["norm_first"] else y * z * sig
    r = 1 / torch.sqrt(torch.linalg.vecdot(v, v)[..., None] / (d // k) + 1e-5)
    if op == "norm":
        out = v * r * w * (z * sig if c["norm_first"] else 1)
        out = out.reshape(b, L, d)
        return out if c["out_order"] == "token" else out.transpose(1, 2)
    g = d64(s["dout"])
    g = (g if c["out_order"] == "token" else g.transpose(1, 2)).reshape(b, L, k, d // k)
    dgate = sig + z * sig * (1 - sig)
    unit = v * r  # the normed values; their gradient is projected off their own direction
    dunit = g * w * (z * sig if c["norm_first"] else 1)
    dv = r * (dunit - unit * torch.linalg.vecdot(dunit, unit)[..., None] / (d // k))
    if c["norm_first"]:
        dy, dz, dw = dv, g * unit * w * dgate, (g * z * sig * unit).sum((0, 1))
    else:
        dy, dz, dw = dv * z * sig, dv * y * dgate, (g * unit).sum((0, 1))
    back = lambda t: t.reshape(b, L, d).transpose(1, 2)  # noqa: E731
    return {"dy": back(dy), "dz": back(dz), "dweight": dw.reshape(-1)}
