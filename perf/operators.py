"""What is measured of the rotary and packed-attention operators: cases, inputs, plain forms.

Three operators, used one after the other by a program that runs attention over tokens of any
lengths:

- ``rope``: rotary positions on queries and keys (rope_fwd), on a line or on the two axes of a
  patch grid, both pair layouts, the whole head or its first part, with scaled frequencies, and
  turned back (inverse).
- ``norm``: the per-head norm of queries and keys with the rotation in the same pass
  (qk_norm_rope_fwd).
- ``attn``: attention over packed sequences of different lengths (packed_attn_fwd), causal or
  not, with grouped heads, from single query tokens against a long cache to whole prompts.

Where ``own`` is false, ``run`` computes them with elementary torch operations in 32 bits (the
angles in 64); where it is true, through this package's entry points.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

# Scaled frequencies: (factor, context the base was made for, low, high).
SCALES = {"none": (1.0, 0, 0.0, 0.0), "linear": (4.0, 0, 0.0, 0.0), "ntk": (8.0, 0, 0.0, 0.0),
          "bands": (8.0, 8192, 1.0, 4.0), "yarn": (16.0, 4096, 1.0, 32.0)}


def listed():
    return [
        # one decoding step of 8 sequences: latency, positions far out, yarn scaling
        dict(name="rope_step", op="rope", batch=0, tokens=8, hq=32, hk=8, d=128, rd=128, axes=1,
             far=131072, inter=False, inverse=False, scale="yarn", dtype="bf16", packed=False),
        # the DeiT-S grid: 64 images of 14 x 14 patches, 6 heads of 64, both axes, written as
        # [B, heads, N, d] for the grid attention that follows
        dict(name="rope_grid", op="rope", batch=64, tokens=196, hq=6, hk=6, d=64, rd=64, axes=2,
             far=14, inter=True, inverse=False, scale="none", dtype="f32", packed=True),
        # cached keys of a long prompt moved to other positions: turned back, part of the head
        dict(name="rope_back", op="rope", batch=0, tokens=6007, hq=8, hk=0, d=128, rd=64, axes=1,
             far=32768, inter=True, inverse=True, scale="bands", dtype="f16", packed=False),
        # a decoding step of 64 sequences
        dict(name="norm_step", op="norm", batch=0, tokens=64, hq=32, hk=8, d=128, rd=128, axes=1,
             far=131072, inter=False, scale="bands", dtype="bf16", packed=True, norm="rms",
             gain="bf16"),
        # images of 56 x 56 patches, 6 heads of 64, layer norms per head
        dict(name="norm_grid", op="norm", batch=8, tokens=3136, hq=6, hk=6, d=64, rd=64, axes=2,
             far=56, inter=False, scale="none", dtype="f16", packed=True, norm="layer",
             gain="f32"),
        # a packed prompt, read out of the projection's output
        dict(name="norm_prompt", op="norm", batch=0, tokens=16384, hq=32, hk=8, d=128, rd=128,
             axes=1, far=16384, inter=False, scale="ntk", dtype="bf16", packed=True, norm="rms",
             gain="bf16"),
        # one decoding step, 32 sequences of very different lengths in a cache of 8192 each
        dict(name="attn_step", op="attn", batch=32, q_lo=1, q_hi=1, k_lo=100, k_hi=8192,
             cache=True, hq=32, hk=8, d=128, causal=True, dtype="bf16", lens=1),
        # one decoding step of a single sequence with a long cache: few rows, one long axis
        dict(name="attn_step_long", op="attn", batch=1, q_lo=1, q_hi=1, k_lo=65000, k_hi=65000,
             cache=True, hq=32, hk=8, d=128, causal=True, dtype="f16", lens=2),
        # a piece of a prompt against what is cached already
        dict(name="attn_piece", op="attn", batch=2, q_lo=509, q_hi=512, k_lo=12000, k_hi=16384,
             cache=True, hq=16, hk=4, d=128, causal=True, dtype="f16", lens=3),
        # prompts of different lengths, causal
        dict(name="attn_prompt", op="attn", batch=8, q_lo=500, q_hi=8192, k_lo=0, k_hi=0,
             cache=False, hq=32, hk=8, d=128, causal=True, dtype="bf16", lens=4),
        # images of many resolutions (up to 56 x 56 patches) packed, 6 heads of 64, all pairs
        dict(name="attn_images", op="attn", batch=48, q_lo=196, q_hi=3136, k_lo=0, k_hi=0,
             cache=False, hq=6, hk=6, d=64, causal=False, dtype="bf16", lens=5),
        # many short sequences, odd head size
        dict(name="attn_short", op="attn", batch=200, q_lo=1, q_hi=190, k_lo=0, k_hi=0,
             cache=False, hq=12, hk=4, d=80, causal=True, dtype="bf16", lens=6),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_rot(rng, op):
    hk = rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([32, 48, 64, 64, 72, 80, 96, 128, 128, 128, 192, 256])
    axes = rng.choice([1, 1, 2])
    rd = d if rng.random() < 0.6 else max(4 * axes, d // rng.choice([2, 4]) // 4 * 4)
    batch = rng.choice([0, 0, rng.randint(1, 32)])
    tokens = _log(rng, 1, 12000)
    if batch:
        tokens = max(1, tokens // batch)
    case = dict(op=op, batch=batch, tokens=tokens, hq=hk * rng.choice([1, 1, 2, 4]), hk=hk, d=d,
                rd=rd, axes=axes, far=_log(rng, 16, 1 << 20) if axes == 1 else rng.randint(4, 200),
                inter=rng.random() < 0.5,
                scale=rng.choice(sorted(SCALES)) if rd // axes >= 16 else "none",
                dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), packed=rng.random() < 0.5)
    if op == "rope":
        case["inverse"] = rng.random() < 0.3
    else:
        case["norm"] = rng.choice(["rms", "rms", "layer"])
        case["gain"] = rng.choice(["f32", case["dtype"]])
    return case


def _draw_attn(rng):
    hk = rng.choice([1, 2, 3, 4, 6, 8])
    hq = hk * rng.choice([1, 1, 2, 3, 4, 8])
    form = rng.choice(["step", "piece", "self", "self"])
    if form == "step":
        q = (1, rng.choice([1, 1, 4]))
        hi = _log(rng, 16, 60000)
        batch = min(64, _log(rng, 1, 262144 // hi + 1))
        k = (max(1, hi // rng.choice([1, 3, 40])), hi)
    elif form == "piece":
        hi = _log(rng, 300, 8192)
        q = (rng.randint(1, 60), rng.randint(64, 300))
        batch = rng.randint(1, 4)
        k = (300, hi)
    else:
        hi = _log(rng, 8, 6000)
        q = (max(1, hi // rng.choice([1, 2, 10, 50])), hi)
        batch = min(128, _log(rng, 1, 24000 // hi + 1))
        k = (0, 0)
    return dict(op="attn", batch=batch, q_lo=q[0], q_hi=q[1], k_lo=k[0], k_hi=k[1],
                cache=form != "self", hq=hq, hk=hk,
                d=rng.choice([32, 64, 64, 80, 96, 128, 128]), causal=rng.random() < 0.7,
                dtype=rng.choice(["bf16", "bf16", "f16"]), lens=rng.randint(10, 10**6))


def draw(rng):
    op = rng.choice(["rope", "norm", "attn", "attn"])
    if op != "attn":
        return _draw_rot(rng, op)
    top = max(work(c)["flops"] for c in listed())
    while True:
        case = _draw_attn(rng)
        if work(case)["flops"] <= top:
            return case


def _lens(case):
    """Query and key lengths of an attention case: log-uniform, from the case alone."""
    rng = random.Random(case["lens"])
    nq = [_log(rng, case["q_lo"], case["q_hi"]) for _ in range(case["batch"])]
    if not case["cache"]:
        return nq, list(nq)
    nk = [_log(rng, case["k_lo"], case["k_hi"]) for _ in range(case["batch"])]
    return nq, nk


def work(case):
    size = 4 if case["dtype"] == "f32" else 2
    if case["op"] != "attn":
        tokens = max(case["batch"], 1) * case["tokens"]
        heads = tokens * (case["hq"] + case["hk"])
        flops = heads * case["rd"] // 2 * 6
        positions = case["tokens"] * case["axes"] * 4
        if case["op"] == "norm":
            flops += heads * case["d"] * 4
        return {"bytes": 2 * heads * case["d"] * size + positions, "flops": flops}
    nq, nk = _lens(case)
    pairs = 0
    for a, b in zip(nq, nk):
        if not case["causal"]:
            pairs += a * b
        else:  # query i sees keys 0 .. i + b - a
            first = max(0, a - b)
            rows = a - first
            pairs += rows * (first + 1 + b - a) + rows * (rows - 1) // 2
    d = case["d"]
    return {"bytes": (2 * sum(nq) * case["hq"] + 2 * sum(nk) * case["hk"]) * d * size,
            "flops": 4 * d * case["hq"] * pairs}


# ---------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(*shape, generator=g, dtype=torch.float32, device=DEV).to(dtype)


def _rot_inputs(case, seed):
    """q, k (token-major, strided when they are parts of one projection's output), positions
    and gains. Channels differ in size, as projections' outputs do."""
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    lead = (case["batch"], case["tokens"]) if case["batch"] else (case["tokens"],)
    hq, hk, d = case["hq"], case["hk"], case["d"]
    spread = torch.exp(0.5 * torch.randn(d, generator=g, device=DEV))
    if case["packed"]:
        x = (torch.randn(*lead, hq + 2 * hk, d, generator=g, device=DEV) * spread).to(dt)
        q, k = x[..., :hq, :], x[..., hq:hq + hk, :]
    else:
        q = (torch.randn(*lead, hq, d, generator=g, device=DEV) * spread).to(dt)
        k = (torch.randn(*lead, hk, d, generator=g, device=DEV) * spread).to(dt) if hk else None
    n, far = case["tokens"], case["far"]
    if case["axes"] == 2:  # patches of a grid far columns wide, row-major
        t = torch.arange(n, device=DEV)
        pos = torch.stack([t // far, t % far], dim=1).to(torch.int32)
    elif n <= 64:  # single tokens of several sequences
        pos = torch.randint(0, far, (n,), generator=g, device=DEV).to(torch.int32)
    else:  # a run of tokens that ends anywhere up to far
        start = int(torch.randint(0, max(1, far - n + 1), (1,), generator=g, device=DEV))
        pos = torch.arange(start, start + n, device=DEV, dtype=torch.int32)
    gains = None
    if case["op"] == "norm":
        gains = [(1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(DTYPES[case["gain"]])
                 for _ in range(2)]
    return q, k, pos, gains


def _attn_inputs(case, seed):
    """q packed; k, v packed, or in a cache of the longest length per sequence."""
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    nq, nk = _lens(case)
    cap = case["k_hi"]
    rows = case["batch"] * cap if case["cache"] else sum(nk)
    q = _normal(g, (sum(nq), case["hq"], case["d"]), dt)
    k = _normal(g, (rows, case["hk"], case["d"]), dt)
    v = _normal(g, (rows, case["hk"], case["d"]), dt)
    starts = [b * cap if case["cache"] else sum(nk[:b]) for b in range(case["batch"])]
    return q, k, v, nq, nk, starts


def _frequencies(case):
    """Radians per position of each pair (64 bits), and the rotation's magnitude."""
    per_axis = case["rd"] // case["axes"]
    factor, ctx, low, high = SCALES[case["scale"]]
    base = 10000.0
    if case["scale"] == "ntk":
        base *= factor ** (per_axis / (per_axis - 2))
    i = torch.arange(per_axis // 2, dtype=torch.float64, device=DEV)
    f = base ** (-2.0 * i / per_axis)
    magnitude = 1.0
    if case["scale"] == "linear":
        f = f / factor
    elif case["scale"] == "bands":
        turns = ctx * f / (2 * math.pi)
        s = ((turns - low) / (high - low)).clamp(0, 1)
        f = f * ((1 - s) / factor + s)
    elif case["scale"] == "yarn":
        def at(turns):  # the index whose pair turns that often over the context
            return per_axis * math.log(ctx / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(0, math.floor(at(high))), min(per_axis - 1, math.ceil(at(low)))
        ramp = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
        f = f / factor * ramp + f * (1 - ramp)
        magnitude = 0.1 * math.log(factor) + 1.0
    return f.repeat(case["axes"]), magnitude


def prepare(case, seed):
    if case["op"] == "attn":
        q, k, v, nq, nk, starts = _attn_inputs(case, seed)
        state = dict(case=case, q=q, k=k, v=v, scale=case["d"] ** -0.5)
        cu_q = [0]
        for n in nq:
            cu_q.append(cu_q[-1] + n)
        if own:
            as_ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
            state["cu_q"] = as_ints(cu_q)
            state["cu_k"] = as_ints(starts + [k.shape[0]])
            state["k_lens"] = as_ints(nk) if case["cache"] else None
        else:
            state["groups"] = _groups(case, nq, nk, cu_q, starts)
        return state
    q, k, pos, gains = _rot_inputs(case, seed)
    state = dict(case=case, q=q, k=k, pos=pos, gains=gains)
    if own:
        import vision_transformer_attention_gb300 as vta
        factor, ctx, low, high = SCALES[case["scale"]]
        state["phases"], state["magnitude"] = vta.rope_build_phases(
            case["rd"], axes=case["axes"], scaling=getattr(vta, "RPE_ROPE_" + case["scale"].upper()),
            factor=factor, context=ctx, low=low, high=high)
    else:
        state["freqs"], state["magnitude"] = _frequencies(case)
    return state


def _groups(case, nq, nk, cu_q, starts):
    """Plain attention's plan: runs of sequences padded to a common length, few enough that
    their scores stay below 4 GB, each with its gather and scatter indices and its mask."""
    groups, b = [], 0
    while b < len(nq):
        e, mq, mk = b, 0, 0
        while e < len(nq):
            tq, tk = max(mq, nq[e]), max(mk, nk[e])
            if e > b and (e + 1 - b) * case["hq"] * tq * tk * 4 > (1 << 32):
                break
            mq, mk, e = tq, tk, e + 1
        i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
        col = lambda x: torch.tensor(x[b:e], device=DEV).view(-1, 1)  # noqa: E731
        lq, lk = col(nq), col(nk)
        rows_q = col(cu_q) + torch.minimum(i, lq - 1)
        rows_k = col(starts) + torch.minimum(j, lk - 1)
        seen = j.view(1, 1, -1) < lk.view(-1, 1, 1)
        if case["causal"]:
            seen = seen & (j.view(1, 1, -1) <= (i + lk - lq).unsqueeze(-1))
        groups.append((rows_q, rows_k, seen, i < lq))
        b = e
    return groups


# ---------------------------------------------------------------- one pass


def _rotate(x, c, s, rd, inter):
    """x [..., heads, d] in 32 bits; c, s [tokens, 1, rd / 2]."""
    if inter:
        a, b = x[..., 0:rd:2], x[..., 1:rd:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :rd // 2], x[..., rd // 2:rd]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., rd:]], dim=-1)


def _plain_rot(state):
    case = state["case"]
    pos = state["pos"].double().reshape(-1, case["axes"])
    angle = pos.repeat_interleave(case["rd"] // 2 // case["axes"], dim=1) * state["freqs"]
    m = state["magnitude"]
    c, s = (angle.cos() * m).float().unsqueeze(1), (angle.sin() * m).float().unsqueeze(1)
    if case["op"] == "rope" and case["inverse"]:
        s = -s
    outs = []
    for t, x in enumerate((state["q"], state["k"])):
        if x is None:
            outs.append(None)
            continue
        y = x.float()
        if case["op"] == "norm":
            if case["norm"] == "layer":
                y = y - y.mean(-1, keepdim=True)
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6) * state["gains"][t].float()
        y = _rotate(y, c, s, case["rd"], case["inter"]).to(x.dtype)
        # batches go on as [B, heads, N, d], where the grid attention reads them
        outs.append(y.transpose(1, 2).contiguous() if case["batch"] else y)
    return tuple(y for y in outs if y is not None)


def _plain_attn(state):
    case, q, k, v = state["case"], state["q"], state["k"], state["v"]
    hq, hk, d = case["hq"], case["hk"], case["d"]
    g = hq // hk
    outs = []
    for rows_q, rows_k, seen, real in state["groups"]:
        n, mq = rows_q.shape
        mk = rows_k.shape[1]
        qs = q[rows_q].float().view(n, mq, hk, g, d).permute(0, 2, 3, 1, 4)
        qs = qs.reshape(n, hk, g * mq, d)
        ks = k[rows_k].float().permute(0, 2, 3, 1)
        vs = v[rows_k].float().permute(0, 2, 1, 3)
        s = (torch.matmul(qs, ks) * state["scale"]).view(n, hk, g, mq, mk)
        s = s.masked_fill_(~seen.unsqueeze(1).unsqueeze(1), -math.inf)
        top = s.amax(-1, keepdim=True)
        p = s.sub_(top.masked_fill(top == -math.inf, 0.0)).exp_()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p.view(n, hk, g * mq, mk), vs).view(n, hk, g, mq, d)
        o = (o / total).masked_fill(total == 0, 0.0)
        outs.append(o.permute(0, 3, 1, 2, 4).reshape(n, mq, hq, d)[real].to(q.dtype))
    return torch.cat(outs)


def run(state):
    case = state["case"]
    if not own:
        return _plain_attn(state) if case["op"] == "attn" else _plain_rot(state)
    import vision_transformer_attention_gb300 as vta
    if case["op"] == "attn":
        return vta.packed_attn_fwd(state["q"], state["k"], state["v"], state["cu_q"],
                                   state["cu_k"], k_lens=state["k_lens"], causal=case["causal"],
                                   scale=state["scale"])
    q, k = state["q"], state["k"]
    outs = {}
    if case["batch"]:  # written as [B, heads, N, d], where the grid attention reads them
        for name, x in (("q_out", q), ("k_out", k)):
            b, n, h, d = x.shape
            outs[name] = torch.empty(b, h, n, d, dtype=x.dtype, device=x.device).transpose(1, 2)
    common = dict(interleaved=case["inter"], magnitude=state["magnitude"], **outs)
    if case["op"] == "rope":
        res = vta.rope_fwd(q, k, state["pos"], state["phases"], inverse=case["inverse"], **common)
    else:
        res = vta.qk_norm_rope_fwd(q, k, state["gains"][0], state["gains"][1], state["pos"],
                                   state["phases"], norm=getattr(vta, "RPE_NORM_" + case["norm"].upper()),
                                   eps=1e-6, **common)
    return tuple(y.transpose(1, 2) if case["batch"] else y for y in res if y is not None)


# ---------------------------------------------------------------- from the definition, in 64 bits


def _exact_rot(case, seed):
    q, k, pos, gains = _rot_inputs(case, seed)
    per_axis = case["rd"] // case["axes"]
    factor, ctx, low, high = SCALES[case["scale"]]
    freqs, magnitude = [], 1.0
    lo_dim = hi_dim = 0.0
    if case["scale"] == "yarn":
        magnitude = 1.0 + math.log(factor) / 10
        # pair i turns ctx * 10000^(-2i / per_axis) / 2 pi times over the context
        lo_dim, hi_dim = (per_axis / 2 * math.log(ctx / 2 / math.pi / t, 10000.0)
                          for t in (high, low))
        lo_dim, hi_dim = max(math.floor(lo_dim), 0), min(math.ceil(hi_dim), per_axis - 1)
    for i in range(per_axis // 2):
        base = 10000.0
        if case["scale"] == "ntk":
            base = base * factor ** (per_axis / (per_axis - 2))
        f = 1.0 / base ** (2 * i / per_axis)
        if case["scale"] == "linear":
            f /= factor
        elif case["scale"] == "bands":
            wave = 2 * math.pi / f
            if wave > ctx / low:
                f /= factor
            elif wave >= ctx / high:
                mix = (ctx / wave - low) / (high - low)
                f = (1 - mix) * f / factor + mix * f
        elif case["scale"] == "yarn":
            keep = 1 - min(1.0, max(0.0, (i - lo_dim) / max(hi_dim - lo_dim, 0.001)))
            f = f * keep + f / factor * (1 - keep)
        freqs.append(f)
    half = case["rd"] // 2
    turn = torch.zeros(case["tokens"], half, dtype=torch.complex128, device=DEV)
    where = pos.to(torch.float64).reshape(-1, case["axes"])
    for p in range(half):
        axis, i = divmod(p, per_axis // 2)
        turn[:, p] = torch.polar(torch.full_like(where[:, axis], magnitude),
                                 where[:, axis] * freqs[i])
    if case.get("inverse"):
        turn = turn.conj()
    outs = []
    for t, x in enumerate((q, k)):
        if x is None:
            continue
        y = x.to(torch.float64)
        if case["op"] == "norm":
            if case["norm"] == "layer":
                y = (y - y.mean(-1, keepdim=True)) / torch.sqrt(
                    y.var(-1, unbiased=False, keepdim=True) + 1e-6)
            else:
                y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + 1e-6)
            y = y * gains[t].to(torch.float64)
        y = y.clone()
        first = slice(0, case["rd"], 2) if case["inter"] else slice(0, half)
        second = slice(1, case["rd"], 2) if case["inter"] else slice(half, case["rd"])
        z = torch.complex(y[..., first].contiguous(), y[..., second].contiguous())
        z = z * turn.unsqueeze(1)
        y[..., first], y[..., second] = z.real, z.imag
        outs.append(y.transpose(1, 2).contiguous() if case["batch"] else y)
    return tuple(outs)


def _exact_attn(case, seed):
    q, k, v, nq, nk, starts = _attn_inputs(case, seed)
    group = case["hq"] // case["hk"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=DEV)
    at = 0
    for b, (a, n) in enumerate(zip(nq, nk)):
        keys = slice(starts[b], starts[b] + n)
        for h in range(case["hq"]):
            kh, vh = (x[keys, h // group].to(torch.float64) for x in (k, v))
            for r in range(0, a, 2048):
                rows = slice(at + r, at + min(a, r + 2048))
                s = q[rows, h].to(torch.float64) @ kh.T / math.sqrt(case["d"])
                if case["causal"]:
                    i = torch.arange(r, min(a, r + 2048), device=DEV).unsqueeze(1)
                    hidden = torch.arange(n, device=DEV).unsqueeze(0) > i + (n - a)
                    s[hidden] = -math.inf
                out[rows, h] = torch.softmax(s, dim=-1).nan_to_num(0.0) @ vh
        at += a
    return out


def exact(case, seed):
    return _exact_attn(case, seed) if case["op"] == "attn" else _exact_rot(case, seed)
