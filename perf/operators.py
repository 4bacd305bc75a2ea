"""What the operators around the semi-CRF loss cost, and what they compute.

Three operators make one training step together with the loss: linear attention
with a decay for each head (features of positions that are too many for quadratic
attention), group norm with an activation on channels-last rows, and AdamW over
many tensors.  A case names one pass through one of them:

  attention  mode forward | training | step; B sequences, T positions, H heads,
             dk/dv widths, type, ragged lengths, state in and out, direction
  norm       mode forward | training; N rows of S positions and C channels, G groups
  adamw      tensors of an encoder of `layers` x `width` and the CRF's tables (labels,
             durations); states in 32 or 8 bits

``own`` False computes the plain forms (elementary torch operations in float32, or
in float64 where a border decides); ``own`` True makes the framework's calls.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


# ---------------------------------------------------------------- cases

def _attention(name, mode, dtype, B, T, H, dk, dv, ragged=False, state=False, reverse=False, packed=False):
    return dict(name=name, op="attention", mode=mode, dtype=dtype, B=B, T=T, H=H, dk=dk, dv=dv, ragged=ragged,
                state=state, reverse=reverse, packed=packed)


def _norm(name, mode, dtype, N, S, C, G, activation, ragged=False):
    return dict(name=name, op="norm", mode=mode, dtype=dtype, N=N, S=S, C=C, G=G, activation=activation,
                ragged=ragged)


def _adamw(name, bits, dtype, layers, width, labels, durations):
    return dict(name=name, op="adamw", bits=bits, dtype=dtype, layers=layers, width=width, labels=labels,
                durations=durations)


def listed():
    return [
        # labelling one live stream, position by position: latency alone
        _attention("step, one stream", "step", "fp32", 1, 1, 4, 64, 64),
        # the same for many streams at once: reads and writes every state
        _attention("step, many streams", "step", "bf16", 256, 1, 8, 128, 128),
        # a batch of sentences of the named-entity workload's lengths
        _attention("attention, sentences", "forward", "fp32", 32, 512, 4, 64, 64, ragged=True),
        # training on the speech workload's utterances
        _attention("attention, speech training", "training", "bf16", 16, 4000, 8, 64, 64, packed=True),
        # one chromosome-scale sequence, read in pieces: state in and out
        _attention("attention, genome", "forward", "bf16", 1, 100_000, 8, 64, 64, state=True),
        # wide heads, backwards in time (the second half of a bidirectional encoder)
        _attention("attention, wide reversed", "forward", "bf16", 4, 20_000, 8, 128, 128, reverse=True),
        # emissions of the named-entity workload, one group over its 17 labels: latency
        _norm("norm, sentences", "forward", "fp32", 32, 512, 17, 1, "none", ragged=True),
        # speech features in training
        _norm("norm, speech training", "training", "fp32", 16, 4000, 128, 8, "silu"),
        # each position on its own, one group for each head, behind the attention
        _norm("norm, positions training", "training", "bf16", 64_000, 1, 512, 8, "silu"),
        # the large-label workload's emissions
        _norm("norm, large", "forward", "bf16", 4, 200_000, 256, 32, "gelu"),
        # an encoder's weights in two types beside the CRF's tables, whose gradients come in float64
        _adamw("adamw, encoder", 32, "bf16", 4, 1280, 256, 512),
        # the same tensors in float32 with states in 8 bits
        _adamw("adamw, encoder 8 bits", 8, "fp32", 4, 1280, 256, 512),
    ]


def _log_between(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["step", "attention", "attention", "norm", "norm", "adamw"])
    dtype = rng.choice(["fp32", "bf16", "bf16", "fp16"])
    if kind == "step":
        return _unnamed(_attention("", "step", dtype, _log_between(rng, 1, 256), 1, rng.randint(1, 8),
                                   rng.randint(8, 128), rng.randint(8, 128)))
    if kind == "attention":
        H, dk = rng.randint(1, 8), rng.choice([rng.randint(8, 128), 64, 32])
        dv = rng.choice([dk, dk, rng.randint(8, 128)])
        mode = rng.choice(["forward", "training"])
        B = _log_between(rng, 1, 32)
        most = (16 * 4000 * 8 * 64) // (B * H * max(dk, dv) * (1 if mode == "training" else 2)) + 1
        T = _log_between(rng, 1, max(2, min(100_000, most)))
        return _unnamed(_attention("", mode, dtype, B, T, H, dk, dv, ragged=rng.random() < 0.5,
                                   state=rng.random() < 0.5, reverse=rng.random() < 0.4,
                                   packed=rng.random() < 0.5))
    if kind == "norm":
        G = rng.choice([1, 2, 4, 8, 16])
        C = G * rng.randint(1, max(1, 512 // G))
        N = _log_between(rng, 1, 64_000)
        S = _log_between(rng, 1, max(1, min(200_000, 32_000_000 // (N * C))))
        return _unnamed(_norm("", rng.choice(["forward", "training"]), dtype, N, S, C, G,
                              rng.choice(["none", "silu", "gelu"]), ragged=rng.random() < 0.5))
    return _unnamed(_adamw("", rng.choice([32, 8]), dtype, rng.randint(0, 4), _log_between(rng, 16, 1200),
                           rng.randint(2, 256), _log_between(rng, 1, 1000)))


def _unnamed(case):
    del case["name"]
    return case


# ---------------------------------------------------------------- inputs

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, dtype=torch.float32, scale=1.0, shift=0.0):
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return x.mul_(scale).add_(shift).to(dtype)


def _lengths(gen, n, most, ragged):
    """Valid positions of each sequence, in [most/2, most] as the named-entity workload draws them."""
    if not ragged:
        return None
    return torch.randint((most + 1) // 2, most + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    return {"attention": _prepare_attention, "norm": _prepare_norm, "adamw": _prepare_adamw}[case["op"]](case, seed)


def _prepare_attention(case, seed):
    gen, dt = _generator(seed), DTYPES[case["dtype"]]
    B, T, H, dk, dv = (case[k] for k in ("B", "T", "H", "dk", "dv"))
    st = dict(case)
    if case["packed"]:                                  # views of one projection's output
        both = _normal(gen, (B, T, H * (2 * dk + dv)), dt)
        st["q"] = both[..., :H * dk].unflatten(-1, (H, dk))
        st["k"] = both[..., H * dk:2 * H * dk].unflatten(-1, (H, dk))
        st["v"] = both[..., 2 * H * dk:].unflatten(-1, (H, dv))
    else:
        st["q"], st["k"], st["v"] = (_normal(gen, (B, T, H, d), dt) for d in (dk, dk, dv))
    # heads forget at rates between one position in 32 and one in 4096
    rate = torch.linspace(5.0, 12.0, H, dtype=torch.float64) if H > 1 else torch.tensor([7.0], dtype=torch.float64)
    st["log_decay"] = torch.log1p(-(2.0 ** -rate)).float().cuda()
    st["lengths"] = _lengths(gen, B, T, case["ragged"])
    st["scale"] = dk ** -0.5
    st["state"] = _normal(gen, (B, H, dk, dv)) if case["state"] or case["mode"] == "step" else None
    if case["mode"] == "step":
        st["q"], st["k"], st["v"] = (st[n][:, 0] for n in ("q", "k", "v"))
    if case["mode"] == "training":
        st["do"] = _normal(gen, (B, T, H, dv), dt)
        st["leaves"] = [st[n].detach().requires_grad_(True) for n in ("q", "k", "v")]
        if st["state"] is not None:
            st["dstate"] = _normal(gen, (B, H, dk, dv))
            st["leaves"].append(st["state"].detach().requires_grad_(True))
    return st


def _prepare_norm(case, seed):
    gen, dt = _generator(seed), DTYPES[case["dtype"]]
    N, S, C = case["N"], case["S"], case["C"]
    st = dict(case)
    offset = _normal(gen, (C,), scale=0.5)
    st["x"] = torch.randn((N, S, C), generator=gen, device="cuda", dtype=dt).add_(offset.to(dt))
    st["weight"] = _normal(gen, (C,), scale=0.1, shift=1.0)
    st["bias"] = _normal(gen, (C,), scale=0.1)
    st["lengths"] = _lengths(gen, N, S, case["ragged"])
    st["eps"] = 1e-5
    if case["mode"] == "training":
        st["dy"] = torch.randn((N, S, C), generator=gen, device="cuda", dtype=dt)
        st["leaves"] = [st[n].detach().requires_grad_(True) for n in ("x", "weight", "bias")]
    return st


def _shapes(case):
    """(shape, parameter type, gradient type) of every tensor of the step."""
    w, C, K = case["width"], case["labels"], case["durations"]
    big, f32, f64 = DTYPES[case["dtype"]], torch.float32, torch.float64
    layer = [((3 * w, w), big, big), ((w, w), big, big), ((w,), f32, f32), ((w,), f32, f32)]
    return layer * case["layers"] + [((C, w), big, big), ((C, C), f32, f64), ((K, C), f32, f64)]


def _prepare_adamw(case, seed):
    gen = _generator(seed)
    st = dict(case, step=100, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
              params=[], grads=[], m=[], v=[], m_scale=None, v_scale=None)
    for shape, pt, gt in _shapes(case):
        st["params"].append(_normal(gen, shape, pt, 0.05))
        st["grads"].append(_normal(gen, shape, scale=1e-3).to(gt))
        st["m"].append(_normal(gen, shape, scale=3e-4))
        st["v"].append(_normal(gen, shape, scale=1e-3).square_())
    if case["bits"] == 8:
        m, v = [_to_8(t.double(), *M8) for t in st["m"]], [_to_8(t.double(), *V8) for t in st["v"]]
        st["m"], st["m_scale"] = [c.view(t.shape) for (c, _), t in zip(m, st["m"])], [s for _, s in m]
        st["v"], st["v_scale"] = [c.view(t.shape) for (c, _), t in zip(v, st["v"])], [s for _, s in v]
    return st


# ---------------------------------------------------------------- one pass

def run(st):
    if st["op"] == "attention":
        return _own_attention(st) if own else _plain_attention(st)
    if st["op"] == "norm":
        return _own_norm(st) if own else _plain_norm(st)
    return _own_adamw(st) if own else _plain_adamw(st)


def _own_attention(st):
    import semi_markov_crf_prefix_b200 as sc
    if st["mode"] == "step":
        o = sc.linear_attention_step(st["q"], st["k"], st["v"], st["log_decay"], st["state"], scale=st["scale"])
        return o, st["state"]
    how = dict(lengths=st["lengths"], scale=st["scale"], reverse=st["reverse"])
    if st["mode"] == "forward":
        if st["state"] is None:
            return (sc.linear_attention(st["q"], st["k"], st["v"], st["log_decay"], **how),)
        return sc.linear_attention(st["q"], st["k"], st["v"], st["log_decay"], initial_state=st["state"],
                                   return_state=True, **how)
    if st["state"] is None:
        o = sc.linear_attention(*st["leaves"], st["log_decay"], **how)
        return (o.detach(), *torch.autograd.grad(o, st["leaves"], st["do"]))
    q, k, v, s0 = st["leaves"]
    o, s1 = sc.linear_attention(q, k, v, st["log_decay"], initial_state=s0, return_state=True, **how)
    return (o.detach(), s1.detach(), *torch.autograd.grad((o, s1), st["leaves"], (st["do"], st["dstate"])))


def _own_norm(st):
    import semi_markov_crf_prefix_b200 as sc
    how = dict(lengths=st["lengths"], eps=st["eps"], activation=st["activation"])
    if st["mode"] == "forward":
        return (sc.group_norm(st["x"], st["G"], st["weight"], st["bias"], **how),)
    x, w, b = st["leaves"]
    y = sc.group_norm(x, st["G"], w, b, **how)
    return (y.detach(), *torch.autograd.grad(y, st["leaves"], st["dy"]))


def _own_adamw(st):
    import semi_markov_crf_prefix_b200 as sc
    st["step"] += 1
    sc.adamw_step(st["params"], st["grads"], st["m"], st["v"], st["step"], lr=st["lr"], betas=st["betas"],
                  eps=st["eps"], weight_decay=st["weight_decay"], exp_avg_scale=st["m_scale"],
                  exp_avg_sq_scale=st["v_scale"])
    if st["bits"] == 32:
        return st["params"], st["m"], st["v"]
    return (st["params"], sc.adamw_state_values(st["m"], st["m_scale"], "exp_avg"),
            sc.adamw_state_values(st["v"], st["v_scale"], "exp_avg_sq"))


# ---------------------------------------------------------------- plain forms

CHUNK = 128


def _valid(lengths, T):
    """[B,T,1,1] truth values, or None where every position counts."""
    if lengths is None:
        return None
    return (torch.arange(T, device="cuda")[None, :] < lengths[:, None])[:, :, None, None]


def _decays(log_decay, n):
    """lambda_h^n in float32 from float64 exponents (n counts positions: up to the whole length)."""
    return torch.exp(log_decay.double().view(-1, *([1] * n.dim())) * n.double()).float()


def _chunked(q, k, v, log_decay, scale, lengths, reverse, state, lead=1):
    """(o, final state) in float32: products inside chunks of 128 positions, one state for each chunk from the
    products of all chunks before it.  Positions behind a sequence's end count nothing.  `lead` is the power of
    lambda that the given state has at the first position."""
    B, T, H, dk = q.shape
    dv, dev = v.shape[-1], q.device
    ok = _valid(lengths, T)
    q, k, v = ((x.float() if ok is None else torch.where(ok, x.float(), 0.0)) for x in (q, k, v))
    L = torch.full((B,), T, device=dev) if lengths is None else lengths.long()
    t = torch.arange(T, device=dev)
    at = (L[:, None] - 1 - t[None, :]) if reverse else t[None, :].expand(B, T)      # position in walking order
    at = at.clamp_min(0)
    # the final state: every key with what is left of it, and the state that was given
    left = (L[:, None] - 1 - at).clamp_min(0)
    w = _decays(log_decay, left).permute(1, 2, 0).unsqueeze(-1)                     # [B,T,H,1]
    final = torch.einsum("bthk,bthv->bhkv", k * w, v)
    if state is not None:
        s0 = state.float()
        final = final + _decays(log_decay, L - 1 + lead).permute(1, 0)[:, :, None, None] * s0
    if reverse:
        q, k, v = q.flip(1), k.flip(1), v.flip(1)
    N = -(-T // CHUNK)
    pad = N * CHUNK - T
    cut = lambda x: torch.nn.functional.pad(x, (0, 0, 0, 0, 0, pad)).view(B, N, CHUNK, H, -1)  # noqa: E731
    q, k, v = cut(q), cut(k), cut(v)
    i = torch.arange(CHUNK, device=dev)
    d = i[:, None] - i[None, :]
    inside = torch.where(d >= 0, _decays(log_decay, d.clamp_min(0)), 0.0)           # [H,c,c]
    p = torch.einsum("bnihk,bnjhk->bnhij", q, k) * inside
    o = torch.einsum("bnhij,bnjhv->bnihv", p, v)
    if N > 1:
        end = _decays(log_decay, CHUNK - 1 - i).transpose(0, 1)[:, :, None]         # [c,H,1]
        s = torch.einsum("bnjhk,bnjhv->bhnkv", k * end, v)
        n = torch.arange(N, device=dev)
        g = n[:, None] - 1 - n[None, :]
        across = torch.where(g >= 0, _decays(log_decay, g.clamp_min(0) * CHUNK), 0.0)
        s = torch.matmul(across, s.reshape(B, H, N, dk * dv)).view(B, H, N, dk, dv)
        o = o + torch.einsum("bnihk,bhnkv->bnihv", q * _decays(log_decay, i + 1).transpose(0, 1)[:, :, None], s)
    o = o.reshape(B, N * CHUNK, H, dv)[:, :T]
    if reverse:
        o, q = o.flip(1), q.reshape(B, N * CHUNK, H, dk)[:, :T].flip(1)
    else:
        q = q.reshape(B, N * CHUNK, H, dk)[:, :T]
    if state is not None:
        w = _decays(log_decay, at + lead).permute(1, 2, 0).unsqueeze(-1)
        o = o + torch.einsum("bthk,bhkv->bthv", q * w, s0)
    o = o * scale
    return (o if ok is None else torch.where(ok, o, 0.0)), final


@torch.no_grad()
def _plain_attention(st):
    q, k, v, ld, scale, s0 = (st[n] for n in ("q", "k", "v", "log_decay", "scale", "state"))
    if st["mode"] == "step":
        s = st["state"]
        s.mul_(torch.exp(ld.double()).float()[None, :, None, None]).add_(k.float()[..., :, None] * v.float()[..., None, :])
        return (q.float()[..., None, :] @ s).squeeze(-2).mul(scale).to(q.dtype), s
    lens, rev = st["lengths"], st["reverse"]
    o, s1 = _chunked(q, k, v, ld, scale, lens, rev, s0)
    out = [o.to(q.dtype)] + ([s1] if s0 is not None else [])
    if st["mode"] == "training":
        do, ds1 = st["do"], st.get("dstate")
        back = lambda s: None if s is None else s.transpose(-1, -2)  # noqa: E731
        dq, _ = _chunked(do, v, k, ld, scale, lens, rev, back(s0))
        # against the direction of time; the state's own gradient arrives behind the last position
        kf, vf, qf, df = k.float(), v.float(), q.float() * scale, do.float()
        dv, ds = _chunked(kf, qf, df, ld, 1.0, lens, not rev, ds1, lead=0)
        dk, _ = _chunked(vf, df, qf, ld, 1.0, lens, not rev, back(ds1), lead=0)
        out += [dq.to(q.dtype), dk.to(q.dtype), dv.to(q.dtype)]
        if s0 is not None:
            # `ds` stands at the first position: the given state is one decay before it
            out.append(ds * torch.exp(ld.double()).float()[None, :, None, None])
    return tuple(out)


def _activate(z, kind):
    if kind == "silu":
        return z / (1.0 + torch.exp(-z))
    if kind == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return z


def _slope(z, kind):
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if kind == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * (2.0 * math.pi) ** -0.5
    return torch.ones_like(z)


@torch.no_grad()
def _plain_norm(st):
    x, G = st["x"], st["G"]
    N, S, C = x.shape
    ok = _valid(st["lengths"], S)
    count = (torch.full((N,), S, device="cuda") if ok is None else st["lengths"]).float()[:, None, None, None] * (C // G)
    g = x.float().view(N, S, G, C // G)
    clear = (lambda z: z) if ok is None else (lambda z: torch.where(ok, z, 0.0))
    total = lambda z: z.sum((1, 3), keepdim=True)  # noqa: E731
    mean = total(clear(g)) / count
    g = clear(g - mean)
    rstd = 1.0 / torch.sqrt(total(g * g) / count + st["eps"])
    g *= rstd
    w, b = st["weight"].view(1, 1, G, -1), st["bias"].view(1, 1, G, -1)
    z = g * w + b
    y = clear(_activate(z, st["activation"])).to(x.dtype).view(N, S, C)
    if st["mode"] == "forward":
        return (y,)
    dz = clear(st["dy"].float().view(N, S, G, -1) * _slope(z, st["activation"]))
    dw, db = (dz * g).sum((0, 1)).view(C), dz.sum((0, 1)).view(C)
    dg = dz * w
    dx = clear(rstd * (dg - total(dg) / count - g * (total(dg * g) / count)))
    return y, dx.to(x.dtype).view(N, S, C), dw, db


# States in 8 bits: blocks of 256 values share a float32 scale (the block's largest magnitude / 1.875); a code is a
# small float of 3 mantissa bits, nearest even.  (exponent bits, bias, sign): first moments 4, 15, yes; second 5, 31, no.
BLOCK = 256
M8, V8 = (4, 15, True), (5, 31, False)


def _blocks(x):
    flat = x.reshape(-1)
    pad = -flat.numel() % BLOCK
    return torch.nn.functional.pad(flat, (0, pad)).view(-1, BLOCK)


def _to_8(x, ebits, bias, signed):
    """(codes [n], scales) of float64 values: borders between codes are decided in float64."""
    n, x = x.numel(), _blocks(x)
    scale = (x.abs().amax(1).float().double() / 1.875).float()
    inverse = torch.where(scale > 0, 1.0 / scale.double(), 0.0)[:, None]
    y = x.abs() * inverse
    e = (torch.frexp(y)[1] - 1).clamp_min(1 - bias)
    code = (e + bias - 1) * 8 + torch.round(torch.ldexp(y, 3 - e)).to(torch.int32)
    code = code.clamp_max((1 << (ebits + 3)) - 1)
    if signed:
        code = code + 128 * (x < 0)
    else:
        code = torch.where((x > 0) & (scale[:, None] > 0), code.clamp_min(1), code)   # what is not zero stays so
    return code.to(torch.uint8).view(-1)[:n].clone(), scale


def _from_8(codes, scale, ebits, bias, signed):
    """float64 values."""
    c = _blocks(codes).int()
    mag = (c & 127) if signed else c
    e = mag >> 3
    val = torch.ldexp(((mag & 7) + 8 * (e > 0)).double(), e.clamp_min(1) - bias - 3) * scale.double()[:, None]
    if signed:
        val = torch.where(c >= 128, -val, val)
    return val.view(-1)[:codes.numel()].view(codes.shape)


def _plain_adamw_one(st, p, g, m, v, ms, vs):
    b1, b2 = st["betas"]
    if st["bits"] == 8:
        g64 = g.double()
        m64 = b1 * _from_8(m, ms, *M8) + (1.0 - b1) * g64
        v64 = b2 * _from_8(v, vs, *V8) + (1.0 - b2) * g64 * g64
        for_p = m64.float(), v64.float()
    else:
        g = g.float()
        for_p = m.mul_(b1).add_((1.0 - b1) * g), v.mul_(b2).add_((1.0 - b2) * g * g)
    c1, c2 = 1.0 - b1 ** st["step"], 1.0 - b2 ** st["step"]
    p.copy_(p.float() * (1.0 - st["lr"] * st["weight_decay"])
            - st["lr"] * (for_p[0] / c1) / (torch.sqrt(for_p[1] / c2) + st["eps"]))
    if st["bits"] == 32:
        return p, m, v
    (cm, s1), (cv, s2) = _to_8(m64, *M8), _to_8(v64, *V8)
    m.copy_(cm.view(m.shape)), ms.copy_(s1), v.copy_(cv.view(v.shape)), vs.copy_(s2)
    return p, _from_8(m, ms, *M8).float(), _from_8(v, vs, *V8).float()


@torch.no_grad()
def _plain_adamw(st):
    st["step"] += 1
    none = [None] * len(st["params"])
    got = [_plain_adamw_one(st, *t) for t in zip(st["params"], st["grads"], st["m"], st["v"], st["m_scale"] or none,
                                                 st["v_scale"] or none)]
    return tuple(list(x) for x in zip(*got))


# ---------------------------------------------------------------- work

def work(case):
    if case["op"] == "attention":
        B, T, H, dk, dv = (case[k] for k in ("B", "T", "H", "dk", "dv"))
        size, state = SIZE[case["dtype"]], B * H * dk * dv * 4
        tokens = B * T * H * (0.75 if case["ragged"] else 1.0)
        if case["mode"] == "step":
            return {"bytes": tokens * (2 * dk + 2 * dv) * size + 2 * state, "flops": tokens * 5 * dk * dv}
        states = 2 * state if case["state"] else 0
        if case["mode"] == "forward":
            # what lies behind a sequence's end is written as zeros
            return {"bytes": (tokens * (2 * dk + dv) + B * T * H * dv) * size + states, "flops": tokens * 4 * dk * dv}
        # q, k, v, do read; o, dq, dk, dv written.  Products: state and output, the three gradients, the
        # state's gradient
        return {"bytes": (tokens * (2 * dk + 2 * dv) + B * T * H * 2 * (dk + dv)) * size + 2 * states,
                "flops": tokens * 12 * dk * dv}
    if case["op"] == "norm":
        n, size = case["N"] * case["S"] * case["C"], SIZE[case["dtype"]]
        read = n * (0.75 if case["ragged"] else 1.0)
        if case["mode"] == "forward":
            return {"bytes": (read + n) * size, "flops": 10 * read}
        return {"bytes": (2 * read + 2 * n) * size, "flops": 30 * read}
    total = 0
    for shape, pt, gt in _shapes(case):
        n = math.prod(shape)
        total += n * (2 * pt.itemsize + gt.itemsize + (16 if case["bits"] == 32 else 4 + 8 + 16 / BLOCK))
    return {"bytes": total, "flops": 14 * sum(math.prod(s) for s, _, _ in _shapes(case))}


# ---------------------------------------------------------------- values in 64 bits

@torch.no_grad()
def exact(case, seed):
    st = prepare(case, seed)
    return {"attention": _exact_attention, "norm": _exact_norm, "adamw": _exact_adamw}[case["op"]](st)


def _exact_attention(st):
    """The sum over pairs of positions itself, in blocks of rows."""
    ld, s0, scale = st["log_decay"].double(), st["state"], st["scale"]
    if st["mode"] == "step":
        q, k, v = (st[n].double() for n in ("q", "k", "v"))
        s = torch.exp(ld)[None, :, None, None] * s0.double() + torch.einsum("bhk,bhv->bhkv", k, v)
        return torch.einsum("bhk,bhkv->bhv", q, s) * scale, s
    q, k, v = (st[n].double().transpose(1, 2) for n in ("q", "k", "v"))            # [B,H,T,d]
    B, H, T, dk = q.shape
    training = st["mode"] == "training"
    do = st["do"].double().transpose(1, 2) if training else None
    if B * H * T * T > 1e11:
        return None
    L = torch.full((B,), T, device="cuda") if st["lengths"] is None else st["lengths"].long()
    t = torch.arange(T, device="cuda")
    ok = (t < L[:, None])[:, None, :, None]
    q, k, v = (torch.where(ok, x, 0.0) for x in (q, k, v))
    if training:
        do = torch.where(ok, do, 0.0)
        dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    o = torch.zeros_like(v)
    rows = max(1, min(T, (1 << 27) // (B * H * T)))
    sign = -1 if st["reverse"] else 1
    for a in range(0, T, rows):
        i = t[a:a + rows]
        lo, hi = (a, T) if st["reverse"] else (0, min(T, a + rows))
        far = sign * (i[:, None] - t[None, lo:hi])
        w = torch.where(far >= 0, torch.exp(ld[:, None, None] * far.clamp_min(0)), 0.0) * scale
        kk, vv = k[:, :, lo:hi], v[:, :, lo:hi]
        p = (q[:, :, a:a + rows] @ kk.transpose(-1, -2)) * w
        o[:, :, a:a + rows] = p @ vv
        if training:
            d = do[:, :, a:a + rows]
            dv_[:, :, lo:hi] += p.transpose(-1, -2) @ d
            dp = (d @ vv.transpose(-1, -2)) * w
            dq[:, :, a:a + rows] = dp @ kk
            dk_[:, :, lo:hi] += dp.transpose(-1, -2) @ q[:, :, a:a + rows]
    at = (L[:, None] - 1 - t) if st["reverse"] else t.expand(B, T)
    since = torch.where(ok, torch.exp(ld[None, :, None, None] * (at + 1)[:, None, :, None]), 0.0)
    left = torch.where(ok, torch.exp(ld[None, :, None, None] * (L[:, None] - 1 - at)[:, None, :, None]), 0.0)
    whole = torch.exp(ld[None, :, None, None] * L[:, None, None, None])
    out = []
    if s0 is not None:
        s0 = s0.double()
        o += (q * since) @ s0 * scale
        s1 = (k * left).transpose(-1, -2) @ v + whole * s0
    if training and s0 is not None:
        ds1 = st["dstate"].double()
        dq += (do * since) @ s0.transpose(-1, -2) * scale
        dk_ += left * (v @ ds1.transpose(-1, -2))
        dv_ += left * (k @ ds1)
        ds0 = (q * since).transpose(-1, -2) @ do * scale + whole * ds1
    out = [o.transpose(1, 2)] + ([s1] if s0 is not None else [])
    if training:
        out += [x.transpose(1, 2) for x in (dq, dk_, dv_)] + ([ds0] if s0 is not None else [])
    return tuple(out)


def _exact_norm(st):
    x, G = st["x"], st["G"]
    N, S, C = x.shape
    training = st["mode"] == "training"
    y, dx = torch.zeros(x.shape, dtype=torch.float64, device="cuda"), None
    w, b = (st[n].double().view(G, -1) for n in ("weight", "bias"))
    if training:
        dx, dw, db = torch.zeros_like(y), torch.zeros_like(w), torch.zeros_like(b)
    rows = max(1, (1 << 26) // (S * C))
    for a in range(0, N, rows):
        u = x[a:a + rows].double().view(-1, S, G, C // G)
        L = (torch.full((N,), S, device="cuda") if st["lengths"] is None else st["lengths"].long())[a:a + rows]
        ok = (torch.arange(S, device="cuda") < L[:, None])[:, :, None, None].double()
        n = L.double()[:, None, None, None] * (C // G)
        mean = (u * ok).sum((1, 3), keepdim=True) / n
        u = u - mean
        r = torch.rsqrt((u * u * ok).sum((1, 3), keepdim=True) / n + st["eps"])
        u = u * r
        z = u * w + b
        kind = st["activation"]
        cdf = 0.5 * torch.erfc(-z / math.sqrt(2.0)) if kind == "gelu" else torch.sigmoid(z) if kind == "silu" else 1.0
        y[a:a + rows] = (z * cdf * ok).view(-1, S, C)
        if training:
            if kind == "gelu":
                slope = cdf + z * torch.exp(-z * z / 2) / math.sqrt(2.0 * math.pi)
            else:
                slope = cdf + z * cdf * (1.0 - cdf)
            dz = st["dy"][a:a + rows].double().view(u.shape) * slope * ok
            dw += (dz * u).sum((0, 1))
            db += dz.sum((0, 1))
            du = dz * w
            back = du - du.sum((1, 3), keepdim=True) / n - u * (du * u).sum((1, 3), keepdim=True) / n
            dx[a:a + rows] = (back * r * ok).view(-1, S, C)
    return (y, dx, dw.view(C), db.view(C)) if training else (y,)


def _nearest_8(x, ebits, bias, signed):
    """The stored values nearest to x, found in the table of all codes' values."""
    n, blocks = x.numel(), _blocks(x)
    scale = (blocks.abs().amax(1).float().double() / 1.875).float().double()[:, None]
    code = torch.arange(1 << (ebits + 3), device="cuda")
    table = torch.where(code < 8, code / 8.0 * 2.0 ** (1 - bias), (1 + (code % 8) / 8.0) * 2.0 ** ((code // 8) - bias).double())
    table = table.double()
    y = torch.where(scale > 0, blocks.abs() / scale, 0.0)
    at = torch.bucketize(y, (table[1:] + table[:-1]) / 2)
    if not signed:
        at = torch.where((blocks > 0) & (scale > 0), at.clamp_min(1), at)
    val = table[at] * scale * (torch.sign(blocks) if signed else 1.0)
    return val.reshape(-1)[:n].view(x.shape)


def _exact_adamw(st):
    b1, b2 = st["betas"]
    t = st["step"] + 1
    params, ms, vs = [], [], []
    for i, (p, g) in enumerate(zip(st["params"], st["grads"])):
        m, v, g = st["m"][i], st["v"][i], g.double()
        if st["bits"] == 8:
            m, v = _from_8(m, st["m_scale"][i], *M8), _from_8(v, st["v_scale"][i], *V8)
        m = m.double() + (1.0 - b1) * (g - m.double())
        v = v.double() + (1.0 - b2) * (g * g - v.double())
        move = m / (1.0 - b1 ** t) / ((v / (1.0 - b2 ** t)).sqrt() + st["eps"])
        params.append(p.double() - st["lr"] * (move + st["weight_decay"] * p.double()))
        ms.append(_nearest_8(m, *M8) if st["bits"] == 8 else m)
        vs.append(_nearest_8(v, *V8) if st["bits"] == 8 else v)
    return params, ms, vs
