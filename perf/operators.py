"""Cases of the gated linear recurrence and of the 8-bit activation checkpoints, with plain forms.

The recurrence of one channel over the tokens t of one sequence, from a state h_0:

    h_t = a_t h_{t-1} + w_t x_t,    y_t = h_t

    gate "log":    a_t = exp(gate_t)               gate "logit": a_t = 1 / (1 + exp(-gate_t))
    input "plain": w_t = 1                         input "complement": w_t = 1 - a_t

and its gradients, with dh_t = dy_t + a_{t+1} dh_{t+1} (the final state's gradient at the end):

    dx_t = w_t dh_t,  dgate_t = a'_t dh_t (h_{t-1} - [complement] x_t),  dh_0 = a_1 dh_1,
    a'_t = a_t ("log") or a_t (1 - a_t) ("logit").

An 8-bit checkpoint holds blocks of 16 consecutive tokens of one channel as int8 codes with one
power-of-two scale: 2^(E - 6) for a block with 2^E <= max|block| < 2^(E + 1), and codes
round(x / scale) within +-127.  A recurrence that trains on checkpoints keeps its x and its gate
(limited to where the decay has not reached its limit: from -16, for logits to 16) that way, and
the exact fp32 state before every span of 64 tokens; its backward pass puts the decoded values in
the place of x and gate, inside each span from that span's exact state.

``run`` computes an operator in its plain form, or (``own``) through the package's calls.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SPAN = 64  # tokens between saved states
BLOCK = 16  # tokens that share one scale in a checkpoint


def listed():
    return [
        # one new token of one sequence, as an interactive decode loop steps it: latency
        dict(name="step one sequence", op="step", b=1, d=4096, dtype="bf16", gate="logit",
             input="complement"),
        # the decode batch of the 8B-shaped layer
        dict(name="step batch 128", op="step", b=128, d=8192, dtype="bf16", gate="log",
             input="plain"),
        # the tiny prefill shape of the tests: one short prompt, fp32
        dict(name="scan tiny", op="scan", b=1, l=256, d=256, dtype="f32", gate="log",
             input="plain", state=True, strided=False),
        # prefill of the 1.3B-shaped layer (64 heads of 64 channels)
        dict(name="scan 1.3B-shaped", op="scan", b=4, l=2048, d=4096, dtype="bf16", gate="log",
             input="plain", state=False, strided=False),
        # long prefill of the 8B-shaped layer (128 heads of 64 channels), the largest pass
        dict(name="scan 8B-shaped", op="scan", b=2, l=16384, d=8192, dtype="bf16", gate="logit",
             input="complement", state=True, strided=False),
        # one very long ragged document on few channels: work only along the time axis
        dict(name="scan long ragged", op="scan", b=1, l=65521, d=1000, dtype="f16", gate="log",
             input="complement", state=True, strided=True),
        # a serving batch of prompts of mixed length, packed, read out of one projection's output
        dict(name="scan packed", op="scan_packed", t=20011, n=22, d=5120, dtype="bf16",
             gate="log", input="plain", strided=True),
        # training step of the 2.7B-shaped layer (80 heads of 64 channels): forward and backward
        dict(name="train 2.7B-shaped", op="train", b=8, l=4096, d=5120, dtype="bf16", gate="log",
             input="plain", state=False),
        # odd sizes in fp32, with the gradient of an initial and of a final state
        dict(name="train odd fp32", op="train", b=3, l=1237, d=777, dtype="f32", gate="logit",
             input="complement", state=True),
        # packed documents of a training batch, state restarting at each
        dict(name="train packed", op="train_packed", t=8191, n=9, d=2560, dtype="f16",
             gate="logit", input="complement", strided=False),
        # the 1.3B-shaped training step that keeps 8-bit checkpoints instead of x and gate
        dict(name="train on checkpoints", op="train_ckpt", b=4, l=2048, d=4096, dtype="bf16",
             gate="log", input="plain", state=False),
        # one layer's activations of a training batch into 8 bits and back
        dict(name="checkpoint round trip", op="ckpt", b=4, l=4096, d=4096, dtype="bf16"),
    ]


def draw(rng):
    def log_int(lo, hi):
        n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        return max(lo, min(hi, n))

    op = rng.choice(["step", "scan", "scan", "scan_packed", "train", "train", "train_packed",
                     "train_ckpt", "ckpt"])
    c = dict(op=op, dtype=rng.choice(["f32", "bf16", "bf16", "f16"]))
    if op != "ckpt":
        c.update(gate=rng.choice(["log", "logit"]), input=rng.choice(["plain", "complement"]))
    if op == "step":
        return dict(c, b=log_int(1, 128), d=log_int(64, 8192))
    most = 1 << 26 if op.startswith("train") else 1 << 27  # elements
    if op.endswith("packed"):
        while True:
            t, d = log_int(64, 32768), log_int(64, 8192)
            if t * d <= most:
                return dict(c, t=t, n=rng.randint(1, 40), d=d, strided=rng.random() < 0.5)
    while True:
        b, d = log_int(1, 8), log_int(64, 8192)
        l = log_int(1, 16384 if op.startswith("train") else 65536)
        if b * l * d <= most:
            break
    c.update(b=b, l=l, d=d)
    if op == "ckpt":
        return c
    c.update(state=rng.random() < 0.5)
    return dict(c, strided=rng.random() < 0.5) if op == "scan" else c


def _activations(gen, lead, d):
    """Two-sided exponential values with a magnitude of its own per channel, 1 % of them x20."""
    dev = gen.device
    x = torch.empty((*lead, d), device=dev).exponential_(generator=gen)
    x *= torch.randint(0, 2, x.shape, device=dev, generator=gen, dtype=torch.int8) * 2 - 1
    scale = 0.25 + torch.rand(d, device=dev, generator=gen)
    return x * torch.where(torch.rand(d, device=dev, generator=gen) < 0.01, 20 * scale, scale)


def _gates(gen, lead, d, form):
    """log: dt A with dt = softplus(N(-2, 0.5)) and A = -exp(U(0, ln 16)) per channel, the decay of
    the framework's own scans; logit: N(2, 1) around a bias per channel."""
    dev = gen.device
    z = torch.randn((*lead, d), device=dev, generator=gen)
    u = torch.rand(d, device=dev, generator=gen)
    if form == "log":
        return -torch.log1p(torch.exp(z * 0.5 - 2)) * torch.exp(u * math.log(16.0))
    return z + 2 + 2 * u


def _lead(c):
    return (c["t"],) if c["op"].endswith("packed") else (c["b"], c["l"])


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "ckpt":
        s["x"] = _activations(gen, (c["b"], c["l"]), c["d"]).to(dt)
        return s
    if c["op"] == "step":
        s["x"] = _activations(gen, (c["b"],), c["d"]).to(dt)
        s["gate"] = _gates(gen, (c["b"],), c["d"], c["gate"]).to(dt)
        s["state"] = torch.randn((c["b"], c["d"]), device="cuda", generator=gen)
        return s
    lead, d = _lead(c), c["d"]
    if c.get("strided"):
        proj = torch.empty((*lead, 2 * d), device="cuda", dtype=dt)  # one projection's output
        s["x"], s["gate"] = proj[..., :d], proj[..., d:]
        s["x"].copy_(_activations(gen, lead, d))
        s["gate"].copy_(_gates(gen, lead, d, c["gate"]))
    else:
        s["x"] = _activations(gen, lead, d).to(dt)
        s["gate"] = _gates(gen, lead, d, c["gate"]).to(dt)
    seqs = c["n"] if c["op"].endswith("packed") else c["b"]
    if c["op"].endswith("packed"):
        # cut points anywhere: lengths from none to many tokens
        cpu = torch.Generator().manual_seed(seed)
        cuts = torch.randint(0, c["t"] + 1, (seqs - 1,), generator=cpu).sort().values
        cu = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([c["t"]])])
        s["cu_seqlens"] = cu.to(torch.int32).cuda()
    if c.get("state", True):
        s["init_state"] = torch.randn((seqs, d), device="cuda", generator=gen)
    if c["op"].startswith("train"):
        s["dy"] = torch.randn((*lead, d), device="cuda", generator=gen).to(dt)
        if c.get("state", True):
            s["dfinal_state"] = torch.randn((seqs, d), device="cuda", generator=gen)
    return s


# ---------------------------------------------------------------------------------------
# plain forms (fp32)
# ---------------------------------------------------------------------------------------
def _decay(gate, form):
    return torch.exp(gate) if form == "log" else torch.sigmoid(gate)


def _weight(gate, form, inp):
    """w: 1, or 1 - a without the cancellation."""
    if inp == "plain":
        return torch.ones_like(gate)
    return -torch.expm1(gate) if form == "log" else torch.sigmoid(-gate)


def _scan(a, b):
    """h_t = a_t h_{t-1} + b_t from h = 0 along the dim before the last, by doubling."""
    n, length = 1, a.shape[-2]
    while n < length:
        b = torch.cat([b[..., :n, :], b[..., n:, :] + a[..., n:, :] * b[..., :-n, :]], -2)
        a = torch.cat([a[..., :n, :], a[..., n:, :] * a[..., :-n, :]], -2)
        n *= 2
    return b


def _first_last(s):
    """Per sequence: whether it holds a token, its first and its last row (rows along dim -2)."""
    cu = s["cu_seqlens"].long()
    return cu[1:] > cu[:-1], cu[:-1], cu[1:] - 1


def _forward(s, x, g, c):
    """(y, h before every token, final states, a, w) in fp32."""
    a, w = _decay(g, c["gate"]), _weight(g, c["gate"], c["input"])
    b = w * x
    if "cu_seqlens" in s:
        full, first, last = _first_last(s)
        init = s["init_state"]
        at = first[full]
        cut = a.clone()
        cut[at] = 0
        b[at] += a[at] * init[full]
        h = _scan(cut, b)
        before = torch.cat([h[:1], h[:-1]])
        before[at] = init[full]
        final = init.clone()
        final[full] = h[last[full]]
        return h, before, final, a, w
    init = s.get("init_state")
    if init is None:
        init = torch.zeros((c["b"], c["d"]), device=x.device)
    b[:, 0] += a[:, 0] * init
    h = _scan(a, b)
    return h, torch.cat([init[:, None], h[:, :-1]], 1), h[:, -1].clone(), a, w


def _backward(s, x, before, a, w, c):
    """(dx, dgate, gradient of the initial states) in fp32."""
    dy = s["dy"].float()
    dfin = s.get("dfinal_state")
    nxt = torch.cat([a[..., 1:, :], torch.zeros_like(a[..., :1, :])], -2)
    if "cu_seqlens" in s:
        full, first, last = _first_last(s)
        end = last[full]
        nxt[end] = 0
        dy = dy.clone()
        dy[end] += dfin[full]
    elif dfin is not None:
        dy = torch.cat([dy[:, :-1], dy[:, -1:] + dfin[:, None]], 1)
    dh = _scan(nxt.flip(-2), dy.flip(-2)).flip(-2)
    da = dh * (before if c["input"] == "plain" else before - x)
    dgate = da * a
    if c["gate"] == "logit":
        dgate = dgate * torch.sigmoid(-s["used_gate"])
    if "cu_seqlens" in s:
        dinit = dfin.clone()
        dinit[full] = a[first[full]] * dh[first[full]]
    else:
        dinit = a[:, 0] * dh[:, 0]
    return w * dh, dgate, dinit


def _rows_of(x, n):
    """[b, l, d] as [b, ceil(l / n), n, d], zeros behind the end."""
    b, l, d = x.shape
    m = -(-l // n)
    if m * n > l:
        x = torch.cat([x, x.new_zeros((b, m * n - l, d))], 1)
    return x.reshape(b, m, n, d)


def _coded(x):
    """(the values that the codes stand for, the biased exponents of the scales) of x [b, l, d]."""
    blocks = _rows_of(x, BLOCK)
    m, e = torch.frexp(blocks.abs().amax(2, keepdim=True))  # largest = m 2^e, m in [0.5, 1)
    e = torch.where(m == 0, -126, torch.clamp(e - 7, min=-126))  # scale 2^e
    q = torch.clamp(torch.round(torch.ldexp(blocks, -e)), -127, 127)
    return torch.ldexp(q, e).reshape(x.shape[0], -1, x.shape[2])[:, :x.shape[1]], (e + 127).squeeze(2)


def _held_gate(g, form):
    return torch.clamp(g, min=-16.0) if form == "log" else torch.clamp(g, -16.0, 16.0)


def _run_plain(s):
    c = s["case"]
    dt = s["x"].dtype
    x = s["x"].float()
    if c["op"] == "ckpt":
        v, e = _coded(x)
        return {"x": v.to(dt), "exponents": e.to(torch.uint8)}
    g = s["gate"].float()
    if c["op"] == "step":
        h = _decay(g, c["gate"]) * s["state"] + _weight(g, c["gate"], c["input"]) * x
        s["state"].copy_(h)
        return {"y": h.to(dt), "state": s["state"]}
    y, before, final, a, w = _forward(s, x, g, c)
    out = {"y": y.to(dt), "final_state": final}
    if not c["op"].startswith("train"):
        return out
    if c["op"] == "train_ckpt":
        x, g = _coded(x)[0], _coded(_held_gate(g, c["gate"]))[0]
        a, w = _decay(g, c["gate"]), _weight(g, c["gate"], c["input"])
        start = before[:, ::SPAN]
        b = _rows_of(w * x, SPAN)
        b[:, :, 0] += _rows_of(a, SPAN)[:, :, 0] * start
        h = _scan(_rows_of(a, SPAN), b)
        before = torch.cat([start[:, :, None], h[:, :, :-1]], 2)
        before = before.reshape(x.shape[0], -1, x.shape[2])[:, :x.shape[1]]
    dx, dgate, dinit = _backward({**s, "used_gate": g}, x, before, a, w, c)
    return {**out, "dx": dx.to(dt), "dgate": dgate.to(dt), "dinit_state": dinit}


# ---------------------------------------------------------------------------------------
# the package's calls
# ---------------------------------------------------------------------------------------
def _run_own(s):
    from quantized_mamba_ssd_b200 import ssd_i8

    c = s["case"]
    x = s["x"]
    if c["op"] == "ckpt":
        q, e = ssd_i8.ssd_i8_ckpt_pack(x)
        return {"x": ssd_i8.ssd_i8_ckpt_unpack(q, e, dtype=c["dtype"]), "exponents": e}
    form = dict(gate_form=c["gate"], input_form=c["input"])
    if c["op"] == "step":
        y = ssd_i8.ssd_i8_gated_step(s["state"], x, s["gate"], **form)
        return {"y": y, "state": s["state"]}
    cu, init = s.get("cu_seqlens"), s.get("init_state")
    packed = cu is not None
    seqs, d = (c["n"] if packed else c["b"]), c["d"]
    final = torch.empty((seqs, d), device=x.device)
    if not c["op"].startswith("train"):
        y = ssd_i8.ssd_i8_gated_scan(x, s["gate"], cu, init_state=init, final_state=final, **form)
        return {"y": y, "final_state": final}
    # what the forward keeps for the backward
    head, length = ((), c["t"]) if packed else ((c["b"],), c["l"])
    spans = torch.empty((*head, -(-length // SPAN), d), device=x.device)
    ckpt = None
    if c["op"] == "train_ckpt":
        ckpt = ssd_i8.ssd_i8_gated_ckpt_empty(x)
    y = ssd_i8.ssd_i8_gated_scan(x, s["gate"], cu, init_state=init, final_state=final,
                                 span_states=spans, ckpt=ckpt, **form)
    dinit = torch.empty((seqs, d), device=x.device)
    states = dict(init_state=init, dfinal_state=s.get("dfinal_state"), dinit_state=dinit, **form)
    if ckpt is not None:
        dx, dgate = ssd_i8.ssd_i8_gated_scan_bwd_ckpt(s["dy"], ckpt, spans, cu, **states)
    else:
        dx, dgate = ssd_i8.ssd_i8_gated_scan_bwd(s["dy"], x, s["gate"], spans, cu, **states)
    return {"y": y, "final_state": final, "dx": dx, "dgate": dgate, "dinit_state": dinit}


def run(state):
    return _run_own(state) if own else _run_plain(state)


def work(case):
    c = case
    e = 4 if c["dtype"] == "f32" else 2
    if c["op"] == "step":
        n = c["b"] * c["d"]
        return {"bytes": n * (3 * e + 8), "flops": 4 * n}  # x, gate, y and the state both ways
    lead = _lead(c) if c["op"] != "ckpt" else (c["b"], c["l"])
    n = math.prod(lead) * c["d"]
    if c["op"] == "ckpt":  # x to codes and scales, codes and scales to x
        blocks = c["b"] * -(-c["l"] // BLOCK) * c["d"]
        return {"bytes": 2 * n * (e + 1) + 2 * blocks, "flops": 3 * n}
    seqs = c["n"] if c["op"].endswith("packed") else c["b"]
    states = seqs * c["d"] * 4 * (2 if c.get("state", True) else 1)  # initial and final
    if not c["op"].startswith("train"):
        return {"bytes": 3 * e * n + states, "flops": 4 * n}  # x, gate, y
    # x, gate, dy; y, dx, dgate; the states and their gradients
    return {"bytes": 6 * e * n + 2 * states, "flops": 14 * n}


# ---------------------------------------------------------------------------------------
# 64 bits, token by token from the definition
# ---------------------------------------------------------------------------------------
def _block_codes(v):
    """The checkpoint's values of one block [b, n, d] in 64 bits, and its scales' exponents."""
    top = v.abs().amax(1)
    k = torch.full_like(top, -126.0)
    some = top > 0
    guess = torch.floor(torch.log2(torch.where(some, top, torch.ones_like(top)))) - 7
    for _ in range(2):  # the exponent whose largest quotient lies in [64, 128)
        guess = torch.where(top * torch.exp2(-guess) >= 128, guess + 1, guess)
    k = torch.where(some, torch.maximum(guess, k), k)
    step = torch.exp2(k)[:, None]
    return torch.round(v / step).clamp(-127, 127) * step, k + 127


def _exact_coded(v):
    vals, exps = zip(*(_block_codes(v[:, t:t + BLOCK]) for t in range(0, v.shape[1], BLOCK)))
    return torch.cat(vals, 1), torch.stack(exps, 1)


def _exact_decay(g, form):
    """a and 1 - a in 64 bits."""
    return (g.exp(), -g.expm1()) if form == "log" else (1 / (1 + (-g).exp()), 1 / (1 + g.exp()))


def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]
    x = s["x"].double()
    if c["op"] == "ckpt":
        v, e = _exact_coded(x)
        return {"x": v, "exponents": e.to(torch.uint8)}
    g = s["gate"].double()
    if c["op"] == "step":
        a, u = _exact_decay(g, c["gate"])
        h = a * s["state"].double() + (x if c["input"] == "plain" else u * x)
        return {"y": h, "state": h}
    cu = s.get("cu_seqlens")
    packed = cu is not None
    if packed:  # one row of tokens; where a sequence begins or ends is looked up by token
        x, g = x[None], g[None]
        offs = cu.tolist()
        begins = {offs[i]: i for i in range(c["n"]) if offs[i + 1] > offs[i]}
        ends = {offs[i + 1] - 1: i for i in range(c["n"]) if offs[i + 1] > offs[i]}
    seqs = c["n"] if packed else c["b"]
    zero = torch.zeros((seqs, c["d"]), dtype=torch.float64, device=x.device)
    init = s["init_state"].double() if "init_state" in s else zero
    a, u = _exact_decay(g, c["gate"])
    length = x.shape[1]
    plain = c["input"] == "plain"
    b = x if plain else u * x
    y, final = torch.empty_like(x), init.clone()
    h = None if packed else init
    for t in range(length):
        if packed and t in begins:
            h = init[begins[t]][None]
        h = a[:, t] * h + b[:, t]
        y[:, t] = h
        if packed and t in ends:
            final[ends[t]] = h[0]
    if not packed:
        final = h
    out = {"y": y[0] if packed else y, "final_state": final}
    if not c["op"].startswith("train"):
        return out
    before = torch.empty_like(x)
    if c["op"] == "train_ckpt":
        lo, hi = -16.0, (math.inf if c["gate"] == "log" else 16.0)
        x, g = _exact_coded(x)[0], _exact_coded(g.clamp(lo, hi))[0]
        a, u = _exact_decay(g, c["gate"])
        b = x if plain else u * x
        for t in range(length):
            if t % SPAN == 0:
                h = y[:, t - 1] if t else init
            before[:, t] = h
            h = a[:, t] * h + b[:, t]
    else:
        before[:, 1:] = y[:, :-1]
        for t, i in (begins.items() if packed else ((0, None),)):
            before[:, t] = init[i] if packed else init
    dy = s["dy"].double()[None] if packed else s["dy"].double()
    dfin = s["dfinal_state"].double() if "dfinal_state" in s else zero
    dx, dgate, dinit = torch.empty_like(x), torch.empty_like(x), dfin.clone()
    back = None if packed else dfin  # the gradient that reaches h_t from behind
    for t in range(length - 1, -1, -1):
        if packed and t in ends:
            back = dfin[ends[t]][None]
        dh = dy[:, t] + back
        back = a[:, t] * dh
        dx[:, t] = dh
        dgate[:, t] = back
        if packed and t in begins:
            dinit[begins[t]] = back[0]
    if not packed:
        dinit = back
    dgate *= before if plain else before - x
    if c["gate"] == "logit":
        dgate *= u
    if not plain:
        dx *= u
    if packed:
        dx, dgate = dx[0], dgate[0]
    return {**out, "dx": dx, "dgate": dgate, "dinit_state": dinit}
