"""Rotary positions and per-head norms (rope_build_phases, rope_fwd,
qk_norm_rope_fwd) against the formulas in 64 bits.

Error allowed of one output y of a pair (x1, x2) with h = |m| hypot(x1, x2)
(after the norm, if there is one): the angle's fraction of a turn is exact but
for its rounding to 24 bits (pi 2^-25), sincospi is good to 2 ulp (2^-23), the
two products, their sum and the magnitude round 2^-24 each: under 2^-21 h. A
norm adds: a sum of up to 256 squares in chains of at most 16 + 5 additions
(21 2^-24, halved by the root), the reciprocal root (2 ulp, 2^-22) and two
products: under 2^-19 h; a layer norm's mean errs by 21 2^-24 of the largest
channel, scaled like the head. The one rounding to the type is half a step,
finfo.eps / 2 of y, or half of its smallest step near zero.
"""
import math

import pytest
import torch

import vision_transformer_attention_gb300 as vta
from vision_transformer_attention_gb300 import _lib, api

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _freqs(rd, axes=1, base=10000.0, scaling=_lib.RPE_ROPE_NONE, factor=1.0, context=0, low=1.0,
           high=32.0):
    """Radians per position of each pair, and the magnitude, from the definitions."""
    D = rd // axes
    out = []
    for i in range(D // 2):
        b = base * factor ** (D / (D - 2)) if scaling == _lib.RPE_ROPE_NTK else base
        f = b ** (-2.0 * i / D)
        if scaling == _lib.RPE_ROPE_LINEAR:
            f /= factor
        elif scaling == _lib.RPE_ROPE_BANDS:
            turns = context * f / (2 * math.pi)
            if turns < low:
                f /= factor
            elif turns <= high:
                s = (turns - low) / (high - low)
                f = (1 - s) * f / factor + s * f
        elif scaling == _lib.RPE_ROPE_YARN:
            at = lambda n: D * math.log(context / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731,B023
            first, last = max(math.floor(at(high)), 0), min(math.ceil(at(low)), D - 1)
            ramp = min(max((i - first) / max(last - first, 0.001), 0.0), 1.0)
            f = f / factor * ramp + f * (1 - ramp)
        out.append(f)
    m = 0.1 * math.log(factor) + 1 if scaling == _lib.RPE_ROPE_YARN else 1.0
    return torch.tensor(out * axes, dtype=torch.float64), m


def _ref(x, pos, freqs, axes, m=1.0, inter=False, inverse=False, norm=None, gain=None, eps=1e-6):
    """(y, allowed error) in 64 bits, on the CPU. x [..., heads, d], pos [..., axes]."""
    t = torch.finfo(x.dtype)
    x = x.detach().cpu().double()
    d, rd = x.shape[-1], 2 * len(freqs)
    slack, mean_err = 2.0 ** -21, 0.0
    if norm is not None:
        slack = 2.0 ** -19
        big = x.abs().amax(-1, keepdim=True)
        if norm == _lib.RPE_NORM_LAYER:
            x = x - x.mean(-1, keepdim=True)
        r = 1 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
        g = torch.ones(d, dtype=torch.float64) if gain is None else gain.detach().cpu().double()
        x = x * r * g
        if norm == _lib.RPE_NORM_LAYER:
            mean_err = 22 * 2.0 ** -24 * big * r * g.abs().max() * abs(m) * math.sqrt(2)
    y, size = x.clone(), x.abs()
    if rd:
        axis = torch.arange(rd // 2) // (rd // 2 // axes)
        ang = pos.cpu().double()[..., axis] * freqs
        c, s = ang.cos().unsqueeze(-2) * m, ang.sin().unsqueeze(-2) * (-m if inverse else m)
        i1 = torch.arange(0, rd, 2) if inter else torch.arange(rd // 2)
        i2 = i1 + 1 if inter else i1 + rd // 2
        y[..., i1] = x[..., i1] * c - x[..., i2] * s
        y[..., i2] = x[..., i2] * c + x[..., i1] * s
        size[..., i1] = size[..., i2] = abs(m) * torch.hypot(x[..., i1], x[..., i2])
    allowed = slack * size + mean_err
    tiny = t.tiny * t.eps / 2
    return y, allowed + t.eps / 2 * (y.abs() + allowed) + tiny


def _check(out, ref):
    y, allowed = ref
    err = (out.detach().cpu().double() - y).abs()
    assert bool((err <= allowed).all()), f"worst {float((err / allowed).max())} of the allowed"


def _randn(*shape, dtype, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype).cuda()


SCALINGS = {
    "none": {}, "linear": dict(scaling=1, factor=4.0), "ntk": dict(scaling=2, factor=8.0),
    "bands": dict(scaling=3, factor=8.0, context=8192, low=1.0, high=4.0),
    "yarn": dict(scaling=4, factor=16.0, context=4096, low=1.0, high=32.0),
}


@pytest.mark.parametrize("name", list(SCALINGS))
@pytest.mark.parametrize("rd,axes", [(128, 1), (64, 2), (2, 1), (12, 2), (256, 1)])
def test_phase_tables(rd, axes, name):
    kw = SCALINGS[name]
    if name == "ntk" and rd // axes < 4:
        pytest.skip("two channels have no other base")
    phases, m = api.rope_build_phases(rd, axes=axes, **kw)
    freqs, want_m = _freqs(rd, axes, **kw)
    assert m == pytest.approx(want_m, rel=1e-7)
    got = (phases.cpu().double() / 2.0 ** 64) % 1.0
    want = (freqs / (2 * math.pi)) % 1.0
    # pow and log to a few ulp of a fraction below 1/6 turn, the table's 2^-53 on reading back
    assert float((got - want).abs().max()) < 2.0 ** -48


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,d,rd,axes", [
    (1, 1, 1, 128, 128, 1), (7, 6, 2, 64, 64, 2), (33, 5, 1, 80, 40, 1), (130, 3, 3, 72, 36, 2),
    (5, 32, 8, 256, 128, 1), (9, 2, 1, 6, 4, 1), (17, 3, 2, 7, 2, 1), (3, 65, 1, 256, 256, 2),
    (611, 4, 2, 96, 96, 1), (4, 2, 2, 255, 4, 1)])
def test_rope_matches_the_formula(tokens, hq, hk, d, rd, axes, inter, dtype):
    q, k = _randn(tokens, hq, d, dtype=dtype, seed=1), _randn(tokens, hk, d, dtype=dtype, seed=2)
    pos = torch.randint(-50, 3000, (tokens, axes), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(3)).cuda()
    phases, m = api.rope_build_phases(rd, axes=axes, **SCALINGS["linear"])
    freqs, _ = _freqs(rd, axes, **SCALINGS["linear"])
    for inverse in (False, True):
        qo, ko = vta.rope_fwd(q, k, pos, phases, interleaved=inter, inverse=inverse,
                              magnitude=1.25)
        for x, y in ((q, qo), (k, ko)):
            _check(y, _ref(x, pos, freqs, axes, 1.25, inter, inverse))


@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("norm", [_lib.RPE_NORM_RMS, _lib.RPE_NORM_LAYER])
@pytest.mark.parametrize("tokens,hq,hk,d,rd,axes,inter,gain", [
    (1, 1, 1, 128, 128, 1, False, "f32"), (50, 6, 6, 64, 64, 2, True, "same"),
    (33, 5, 1, 80, 40, 1, False, None), (130, 3, 3, 72, 36, 2, True, "f32"),
    (6, 32, 8, 128, 0, 1, False, "same"), (9, 2, 1, 7, 2, 1, False, "f32"),
    (5, 3, 1, 256, 64, 1, True, "same"), (4, 1, 2, 1, 0, 1, False, "f32")])
def test_norm_and_rope_match_the_formula(tokens, hq, hk, d, rd, axes, inter, gain, norm, dtype):
    q, k = (_randn(tokens, h, d, dtype=dtype, seed=4 + h) * 3 + 0.5 for h in (hq, hk))
    pos = torch.randint(0, 100000, (tokens, axes), dtype=torch.int32,
                        generator=torch.Generator().manual_seed(5)).cuda()
    gains = [None, None] if gain is None else [
        _randn(d, dtype=F32 if gain == "f32" else dtype, seed=8 + i) for i in range(2)]
    phases = freqs = None
    if rd:
        phases, _ = api.rope_build_phases(rd, axes=axes)
        freqs, _ = _freqs(rd, axes)
    qo, ko = vta.qk_norm_rope_fwd(q, k, *gains, positions=pos if rd else None, phases=phases,
                                  norm=norm, eps=1e-5, interleaved=inter)
    for x, y, g in ((q, qo, gains[0]), (k, ko, gains[1])):
        _check(y, _ref(x, pos, [] if freqs is None else freqs, axes, 1.0, inter, False, norm, g,
                       1e-5))


def test_far_positions_turn_exactly():
    # the last positions of 32 bits: a turn formed in 32 bits would be random here
    phases, _ = api.rope_build_phases(64)
    freqs, _ = _freqs(64)
    pos = torch.tensor([0, 1, -1, 2 ** 24 + 1, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32).cuda()
    x = _randn(6, 2, 64, dtype=F32, seed=9)
    out, none = api.rope_fwd(x, None, pos, phases)
    assert none is None
    y, allowed = _ref(x, pos[:, None], freqs, 1)
    # the table's error, 2^-52 f / 2 pi turns per position, and pow's few ulp of it
    far = pos.cpu().double().abs() * 2.0 ** -49 * x.cpu().double().abs().amax()
    _check(out, (y, allowed + far[:, None, None]))


@pytest.mark.parametrize("V,offset,stride", [(8, 0, 8), (4, 4, 4), (2, 2, 2), (1, 1, 3)])
def test_parts_of_a_projection_and_in_place(V, offset, stride):
    # q and k inside one [tokens, (hq + 2 hk) d] buffer at any offset and row length, turned in
    # place: v, the rows' padding and what lies before stay as they were
    tokens, hq, hk, d = 37, 4, 2, 64
    row = (hq + 2 * hk) * d + stride
    for dtype in (BF16, F32):
        buf = _randn(offset + tokens * row, dtype=dtype, seed=10)
        before = buf.clone()
        x = torch.as_strided(buf, (tokens, hq + 2 * hk, d), (row, d, 1), offset)
        q, k = x[:, :hq], x[:, hq:hq + hk]
        pos = torch.arange(tokens, dtype=torch.int32, device="cuda")
        phases, _ = api.rope_build_phases(d)
        freqs, _ = _freqs(d)
        want = [_ref(t, pos[:, None], freqs, 1) for t in (q, k)]
        out = api.rope_fwd(q, k, pos, phases, q_out=q, k_out=k)
        assert out[0] is q and out[1] is k
        _check(q, want[0])
        _check(k, want[1])
        touched = torch.zeros_like(buf, dtype=torch.bool)
        torch.as_strided(touched, (tokens, hq + hk, d), (row, d, 1), offset).fill_(True)
        assert torch.equal(buf[~touched], before[~touched])


@pytest.mark.parametrize("shared", [True, False])
def test_batches_into_the_grid_layout(shared):
    # [B, N, heads, d] in, [B, heads, N, d] out (what rpe_attn_fwd reads), grid positions
    B, H, W, heads, d = 3, 5, 7, 6, 64
    N = H * W
    x = _randn(B, N, 3 * heads, d, dtype=BF16, seed=11)
    q, k = x[:, :, :heads], x[:, :, heads:2 * heads]
    t = torch.arange(N)
    pos = torch.stack([t // W, t % W], 1).to(torch.int32)
    if not shared:
        pos = torch.stack([pos + 10 * b for b in range(B)])
    pos = pos.cuda()
    phases, _ = api.rope_build_phases(d, axes=2)
    freqs, _ = _freqs(d, 2)
    outs = [torch.empty(B, heads, N, d, dtype=BF16, device="cuda") for _ in range(2)]
    api.qk_norm_rope_fwd(q, k, None, None, pos, phases, norm=_lib.RPE_NORM_LAYER,
                         q_out=outs[0].transpose(1, 2), k_out=outs[1].transpose(1, 2))
    for src, out in zip((q, k), outs):
        _check(out.transpose(1, 2), _ref(src, pos, freqs, 2, norm=_lib.RPE_NORM_LAYER))


def test_inverse_is_the_gradient():
    # y(x) is linear, so its gradient for a cotangent w is the turn back of w; checked against
    # autograd of the formula and against differences of the operator itself
    tokens, heads, d, rd = 11, 3, 64, 32
    x, w = _randn(tokens, heads, d, dtype=F32, seed=12), _randn(tokens, heads, d, dtype=F32, seed=13)
    pos = torch.arange(0, 70 * tokens, 70, dtype=torch.int32, device="cuda")
    phases, m = api.rope_build_phases(rd, **SCALINGS["yarn"])
    freqs, _ = _freqs(rd, **SCALINGS["yarn"])
    grad, _ = api.rope_fwd(w, None, pos, phases, inverse=True, magnitude=m)
    xd = x.cpu().double().requires_grad_(True)
    ang = pos.cpu().double()[:, None, None] * freqs
    a, b = xd[..., :rd // 2], xd[..., rd // 2:rd]
    y = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1) * m
    (torch.cat([y, xd[..., rd:]], -1) * w.cpu().double()).sum().backward()
    ref = xd.grad
    assert float((grad.cpu().double() - ref).abs().max()) < 2.0 ** -20 * float(ref.abs().max()) * 2
    e = _randn(tokens, heads, d, dtype=F32, seed=14)
    hi, _ = api.rope_fwd(x + e, None, pos, phases, magnitude=m)
    lo, _ = api.rope_fwd(x - e, None, pos, phases, magnitude=m)
    diff = ((hi.double() - lo.double()) * w.double()).sum() / 2
    size = (e.double().abs() * w.double().abs()).sum()
    assert abs(float(diff - (grad.double() * e.double()).sum())) < 2.0 ** -18 * float(size) * m


def test_nan_and_infinity_stay_in_their_pair_and_head():
    x = _randn(4, 3, 64, dtype=F16, seed=15)
    x[1, 1, 5] = float("nan")
    x[2, 0, 60] = float("inf")
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    phases, _ = api.rope_build_phases(48)
    y, _ = api.rope_fwd(x, None, pos, phases)
    bad = torch.nonzero(~torch.isfinite(y.float())).tolist()
    assert bad == [[1, 1, 5], [1, 1, 29], [2, 0, 60]]
    y, _ = api.qk_norm_rope_fwd(x, None, None, None, pos, phases)
    bad = {tuple(i[:2]) for i in torch.nonzero(~torch.isfinite(y.float())).tolist()}
    assert bad == {(1, 1), (2, 0)}


def test_no_tokens_and_capture():
    phases, _ = api.rope_build_phases(64)
    empty = torch.empty(0, 4, 64, dtype=BF16, device="cuda")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    assert api.rope_fwd(empty, empty, none, phases)[0].shape == (0, 4, 64)
    x = _randn(20, 4, 64, dtype=BF16, seed=16)
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    out = torch.zeros_like(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        table, _ = api.rope_build_phases(64)
        api.rope_fwd(x, None, pos, table, q_out=out)
    x.copy_(_randn(20, 4, 64, dtype=BF16, seed=17))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, api.rope_fwd(x, None, pos, phases)[0])


def test_python_refusals():
    x = torch.zeros(5, 2, 64, dtype=BF16, device="cuda")
    pos = torch.zeros(5, dtype=torch.int32, device="cuda")
    phases, _ = api.rope_build_phases(64)
    for bad, err in (
            (lambda: api.rope_fwd(x.double(), None, pos, phases), TypeError),
            (lambda: api.rope_fwd(x.cpu(), None, pos, phases), ValueError),
            (lambda: api.rope_fwd(x, x.half(), pos, phases), TypeError),
            (lambda: api.rope_fwd(x, x[:4], pos, phases), ValueError),
            (lambda: api.rope_fwd(x, None, pos.long(), phases), TypeError),
            (lambda: api.rope_fwd(x, None, pos[:4], phases), ValueError),
            (lambda: api.rope_fwd(x, None, pos, None), ValueError),
            (lambda: api.rope_fwd(x.transpose(1, 2), None, pos, phases), ValueError),
            (lambda: api.rope_fwd(x[..., :32], None, pos, phases), vta.RpeError),
            (lambda: api.rope_fwd(x, None, pos, phases, q_out=x[:4]), ValueError),
            (lambda: api.rope_fwd(x, None, pos, phases, q_out=x[:1].expand(5, 2, 64)),
             vta.RpeError),
            (lambda: api.qk_norm_rope_fwd(x, None, torch.ones(64, device="cuda").half(), None),
             TypeError),
            (lambda: api.qk_norm_rope_fwd(x, None, torch.ones(32, device="cuda"), None),
             ValueError),
            (lambda: api.qk_norm_rope_fwd(x, None, None, None, norm=2), vta.RpeError),
            (lambda: api.rope_build_phases(63), vta.RpeError),
            (lambda: api.rope_build_phases(64, base=1.0), vta.RpeError)):
        with pytest.raises(err):
            bad()
