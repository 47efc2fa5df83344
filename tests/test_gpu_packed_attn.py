"""Attention over packed sequences (packed_attn_fwd) against the definition in
64 bits.

Error allowed of an output with W = sum_j softmax_j |v_j| (u: half a step of the
type, finfo.eps / 2): the probabilities' rounding u W, the output's u |out|,
and e W twice (numerator and denominator) for the relative error e of a
probability in fp32: 2^-22 of the exponential, the exponent's rounding (2^-23
of its size, times ln 2), and the score's sum of d products in fp32, where each
addition may lose 2^-23 of the sum of absolute products. lse errs by e.
"""
import math

import pytest
import torch

import vision_transformer_attention_gb300 as vta
from vision_transformer_attention_gb300 import api

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.rpe_device_status(clear=True)
    yield
    assert api.rpe_device_status(clear=True) == 0


def _randn(*shape, dtype=BF16, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return torch.tensor(out, dtype=torch.int32, device="cuda")


def _ref(q, k, v, q_rows, k_rows, causal, scale):
    """(out, allowed, lse, allowed) for one sequence: rows of q, k, v given as slices."""
    qs, ks, vs = (x[r].double().transpose(0, 1) for x, r in ((q, q_rows), (k, k_rows), (v, k_rows)))
    group = qs.shape[0] // ks.shape[0]
    ks, vs = ks.repeat_interleave(group, 0), vs.repeat_interleave(group, 0)
    nq, nk, d = qs.shape[1], ks.shape[1], qs.shape[2]
    s = qs @ ks.transpose(1, 2) * scale
    absolute = qs.abs() @ ks.abs().transpose(1, 2) * scale
    if causal:
        hidden = (torch.arange(nk, device="cuda")[None] >
                  torch.arange(nq, device="cuda")[:, None] + nk - nq)
        s = s.masked_fill(hidden, -math.inf)
        absolute = absolute.masked_fill(hidden, 0.0)
    if nk == 0:
        zero = torch.zeros_like(qs)
        return (zero.transpose(0, 1), zero.transpose(0, 1),
                torch.full((nq, qs.shape[0]), -math.inf, device="cuda").double(), 0.0)
    lse = torch.logsumexp(s, -1)
    p = (s - lse.masked_fill(lse == -math.inf, 0.0).unsqueeze(-1)).exp()
    out, weight = p @ vs, p @ vs.abs()
    e = 2.0 ** -21 + 2.0 ** -22 * absolute.amax(-1) + d * 2.0 ** -23 * absolute.amax(-1)
    u = torch.finfo(q.dtype).eps / 2
    tiny = torch.finfo(q.dtype).tiny * u  # results below the normal range
    allowed = (u + 2 * e.unsqueeze(-1)) * weight + u * out.abs() + tiny
    return (out.transpose(0, 1), allowed.transpose(0, 1), lse.transpose(0, 1),
            (e + 2.0 ** -22 * lse.abs().masked_fill(lse == -math.inf, 0)).transpose(0, 1))


def _check(q, k, v, nq, nk, q0, k0, out, lse, causal, scale):
    for b in range(len(nq)):
        rows = slice(q0[b], q0[b] + nq[b])
        y, ya, z, za = _ref(q, k, v, rows, slice(k0[b], k0[b] + nk[b]), causal, scale)
        err = (out[rows].double() - y).abs()
        assert bool((err <= ya).all()), (
            f"sequence {b} ({nq[b]} queries, {nk[b]} keys): "
            f"worst {float((err / ya.clamp_min(1e-30)).max()):.2f} of the allowed")
        got = lse[rows].double()
        same = (got == z) | ((got - z).abs() <= za)
        assert bool(same.all()), f"sequence {b}: lse"


def _run(nq, nk, hq, hkv, d, causal, dtype, seed=0, capacity=None, scale=None, spread=1.0):
    """Packed queries; keys packed, or in a cache of `capacity` rows each."""
    total_q = sum(nq)
    q0 = _cu(nq).tolist()
    if capacity is None:
        k0, total_k, k_lens = _cu(nk).tolist(), sum(nk), None
        cu_k = _cu(nk)
    else:
        k0 = [b * capacity for b in range(len(nk) + 1)]
        total_k, cu_k = len(nk) * capacity, torch.tensor(k0, dtype=torch.int32, device="cuda")
        k_lens = torch.tensor(nk, dtype=torch.int32, device="cuda")
    q = _randn(total_q, hq, d, dtype=dtype, seed=seed + 1, scale=spread)
    k = _randn(total_k, hkv, d, dtype=dtype, seed=seed + 2)
    v = _randn(total_k, hkv, d, dtype=dtype, seed=seed + 3)
    if capacity is not None:  # what lies behind a sequence's keys must not matter
        for b, n in enumerate(nk):
            k[k0[b] + n:k0[b + 1]] = float("nan")
            v[k0[b] + n:k0[b + 1]] = float("inf")
    out, lse = vta.packed_attn_fwd(q, k, v, _cu(nq), cu_k, k_lens=k_lens, causal=causal, scale=scale,
                                   return_lse=True)
    _check(q, k, v, nq, nk, q0, k0, out, lse, causal, d ** -0.5 if scale is None else scale)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(1, 1, 64), (2, 2, 128), (6, 2, 80), (8, 1, 32), (5, 1, 128),
                                      (7, 7, 8), (128, 1, 64)])
def test_one_sequence(hq, hkv, d, causal, dtype):
    for n in (1, 17, 128, 129, 300):
        _run([n], [n], hq, hkv, d, causal, dtype, seed=n)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (3, 3, 128), (6, 2, 96), (12, 4, 80)])
def test_ragged_sequences(hq, hkv, d, causal):
    # lengths around the tile's, zeros among them, first and last
    nq = [0, 1, 127, 128, 129, 0, 255, 257, 64, 700, 3, 0]
    _run(nq, nq, hq, hkv, d, causal, BF16, seed=20)
    nk = [5, 0, 1, 300, 128, 7, 129, 256, 1000, 640, 0, 2]  # some queries see no key
    _run(nq, nk, hq, hkv, d, causal, F16, seed=21)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (4, 4, 64), (6, 1, 72), (16, 1, 128)])
def test_single_tokens_against_a_cache(hq, hkv, d, causal, dtype):
    nk = [1, 2, 127, 128, 129, 0, 1000, 2048, 511, 1919]
    _run([1] * len(nk), nk, hq, hkv, d, causal, dtype, seed=30, capacity=2048)


@pytest.mark.parametrize("nq,nk,hq,hkv,d", [
    ([1], [20011], 8, 2, 128), ([4], [9000], 4, 1, 64), ([1], [70000], 1, 1, 128),
    ([130, 1, 33], [3000, 4097, 5000], 8, 4, 128), ([509, 512], [3500, 4000], 16, 4, 128),
    ([1, 0, 2], [1, 3000, 0], 2, 2, 64)])
def test_few_queries_against_long_keys(nq, nk, hq, hkv, d):
    for causal in (False, True):
        _run(nq, nk, hq, hkv, d, causal, BF16, seed=40, capacity=max(nk) + 3)
        _run(nq, nk, hq, hkv, d, causal, F16, seed=41)


def test_many_sequences():
    # more sequences than threads of a CTA; empty ones in runs
    g = torch.Generator().manual_seed(50)
    nq = torch.randint(0, 40, (1500,), generator=g).tolist()
    nq[200:300] = [0] * 100
    _run(nq, nq, 4, 2, 64, True, BF16, seed=50)
    nk = torch.randint(0, 300, (900,), generator=g).tolist()
    _run([1] * 900, nk, 4, 1, 128, True, BF16, seed=51, capacity=300)


def test_long_prompt():
    _run([5000, 2100], [5000, 2100], 4, 2, 128, True, BF16, seed=60)
    _run([3137, 196, 2500], [3137, 196, 2500], 3, 3, 64, False, BF16, seed=61)


@pytest.mark.parametrize("spread", [40.0, 0.0])
def test_large_and_equal_scores(spread):
    # rows whose maximum moves by more than 2^8 again and again, and equal scores
    _run([200, 300], [200, 300], 2, 1, 64, True, F16, seed=70, spread=spread)
    _run([1, 2], [3000, 2000], 2, 1, 64, False, F16, seed=71, spread=spread)


def test_growing_scores_rescale_every_tile():
    n, d = 1024, 64
    q = torch.ones(n, 1, d, device="cuda", dtype=F16)
    k = (torch.arange(n, device="cuda") / 64.0)[:, None, None].expand(n, 1, d).to(F16).contiguous()
    v = _randn(n, 1, d, dtype=F16, seed=80)
    for nq in (n, 1):
        out, lse = vta.packed_attn_fwd(q[:nq], k, v, _cu([nq]), _cu([n]), scale=1.0, return_lse=True)
        _check(q, k, v, [nq], [n], [0], [0], out, lse, False, 1.0)


def test_rows_of_no_sequence_stay():
    q, k, v = (_randn(300, 4, 64, seed=90 + i) for i in range(3))
    cu = torch.tensor([10, 60, 60, 201], dtype=torch.int32, device="cuda")
    out = torch.full((300, 4, 64), 7.0, dtype=BF16, device="cuda")
    api.packed_attn_fwd(q, k, v, cu, causal=True, out=out)
    assert bool((out[:10] == 7).all()) and bool((out[201:] == 7).all())
    assert not bool((out[10:201] == 7).all(-1).any())
    # one row per sequence, far apart: the pieces' join leaves the others alone too
    long_k, long_v = (_randn(5000, 4, 64, seed=95 + i) for i in range(2))
    cu = torch.tensor([2, 3, 3], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, 5000, 5000], dtype=torch.int32, device="cuda")
    out.fill_(7.0)
    api.packed_attn_fwd(q[:8], long_k, long_v, cu, cu_k, out=out[:8])
    assert bool((out[:2] == 7).all()) and bool((out[3:] == 7).all())
    assert not bool((out[2] == 7).all(-1).any())


def test_strided_views():
    # q, k, v inside one projection's output; out inside a wider buffer; heads-major memory
    n, hq, hkv, d = 333, 6, 2, 64
    x = _randn(n, hq + 2 * hkv + 1, d, seed=100)
    q, k, v = x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:hq + 2 * hkv]
    wide = torch.zeros(n, hq + 3, d, dtype=BF16, device="cuda")
    out, lse = api.packed_attn_fwd(q, k, v, _cu([100, 233]), causal=True, out=wide[:, 2:2 + hq],
                                   return_lse=True)
    _check(q, k, v, [100, 233], [100, 233], [0, 100], [0, 100], out, lse, True, d ** -0.5)
    assert bool((wide[:, :2] == 0).all()) and bool((wide[:, 2 + hq:] == 0).all())
    q, k, v = (_randn(h, n, d, seed=101 + h).transpose(0, 1) for h in (hq, hkv, hkv))
    out = torch.empty(hq, n, d, dtype=BF16, device="cuda").transpose(0, 1)
    out, lse = api.packed_attn_fwd(q, k, v, _cu([n]), out=out, return_lse=True)
    _check(q, k, v, [n], [n], [0], [0], out, lse, False, d ** -0.5)


def test_values_behind_a_sequence_do_not_matter():
    # the next sequence's NaN and infinities lie in the same key tile
    nq = [100, 50, 60]
    q, k, v = (_randn(210, 2, 128, seed=110 + i) for i in range(3))
    clean = api.packed_attn_fwd(q, k, v, _cu(nq), causal=True)
    k[100:150] = float("nan")
    v[100:150] = float("inf")
    q[100:150] = float("nan")
    out = api.packed_attn_fwd(q, k, v, _cu(nq), causal=True)
    assert torch.equal(out[:100], clean[:100]) and torch.equal(out[150:], clean[150:])
    assert not bool(torch.isfinite(out[100:150].float()).any())


def test_streams_workspaces_and_graphs():
    cases = []
    for seed, nk in ((120, 4000), (121, 6000)):
        q, k, v = _randn(2, 8, 128, seed=seed), _randn(nk, 2, 128, seed=seed + 10), _randn(
            nk, 2, 128, seed=seed + 20)
        cu_q, cu_k = _cu([1, 1]), _cu([nk // 3, nk - nk // 3])
        cases.append((q, k, v, cu_q, cu_k))
    want = [api.packed_attn_fwd(*c) for c in cases]
    # two calls at once on two streams, each with its own workspace
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for c, st in zip(cases, streams):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(20):
                got = api.packed_attn_fwd(*c)
            outs.append(got)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # captured, replayed with other inputs
    c = cases[0]
    out = torch.empty_like(c[0])
    size = api.packed_attn_workspace(2, 4000, 2, 8, 2, 128)
    assert size > 0
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.packed_attn_fwd(*c, out=out, workspace=ws)
    c[0].copy_(cases[1][0])
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, api.packed_attn_fwd(*c))


def test_lengths_outside_the_tensors_set_the_status():
    q, k, v = (_randn(64, 2, 64, seed=130 + i) for i in range(3))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    good = ints(0, 32, 64)
    for cu_q, cu_k, k_lens in ((ints(0, 32, 65), good, None), (ints(-1, 32, 64), good, None),
                               (ints(0, 40, 32), good, None), (good, ints(0, 32, 1 << 30), None),
                               (good, good, ints(33, 1)), (good, good, ints(-1, 1))):
        api.packed_attn_fwd(q, k, v, cu_q, cu_k, k_lens=k_lens)
        assert api.rpe_device_status(clear=True) == 1 << 6
    # overlapping sequences, more of them than the workspace has room for
    long = _randn(6000, 2, 64, seed=135)
    cu_q = torch.tensor([0, 64] * 40, dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0] * 79 + [6000], dtype=torch.int32, device="cuda")
    api.packed_attn_fwd(q, long, long, cu_q, cu_k)
    assert api.rpe_device_status(clear=True) == 1 << 6


def test_python_refusals():
    q = torch.zeros(8, 4, 64, dtype=BF16, device="cuda")
    cu = _cu([8])
    for bad, err in (
            (lambda: api.packed_attn_fwd(q.float(), q.float(), q.float(), cu), vta.RpeError),
            (lambda: api.packed_attn_fwd(q, q.half(), q, cu), TypeError),
            (lambda: api.packed_attn_fwd(q, q, q[:4], cu), ValueError),
            (lambda: api.packed_attn_fwd(q, q[..., :32], q[..., :32], cu), ValueError),
            (lambda: api.packed_attn_fwd(q, q[:, :3], q[:, :3], cu), vta.RpeError),
            (lambda: api.packed_attn_fwd(q, q, q, cu.long()), TypeError),
            (lambda: api.packed_attn_fwd(q, q, q, cu, _cu([4, 4])), ValueError),
            (lambda: api.packed_attn_fwd(q, q, q, cu, k_lens=_cu([1])), ValueError),
            (lambda: api.packed_attn_fwd(q, q, q, cu, scale=0.0), vta.RpeError),
            (lambda: api.packed_attn_fwd(q, q[:, :1].expand(8, 4, 64), q, cu), vta.RpeError),
            (lambda: api.packed_attn_fwd(q[..., :60], q[..., :60], q[..., :60], cu), vta.RpeError),
            (lambda: api.packed_attn_fwd(q, q, q, cu, out=q[:4]), ValueError)):
        with pytest.raises(err):
            bad()
