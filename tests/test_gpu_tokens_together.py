"""The calls on tokens as a program uses them, one after another: a projection's queries and keys
normed and turned in place or into a cache, attention over them, prompts and then single tokens,
captured steps, and the patch grid's attention behind the rotation. Each stage is held to its own
tolerance on the tensors that it read (test_gpu_rope, test_gpu_packed_attn). And what both kinds of
call share: the quick way into the library against the checked one, and offsets past 2^31.
"""
import random

import pytest
import torch

from test_gpu_packed_attn import BF16, F16, _check as check_attn, _cu, _randn, _ref as ref_attn, _run
from test_gpu_rope import _check as check_rope, _freqs, _ref as ref_rope
from vision_transformer_attention_gb300 import _lib, api, workloads

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    api.rpe_device_status(clear=True)
    yield
    assert api.rpe_device_status(clear=True) == 0


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Layer:
    """One attention layer over a cache: projection, norm and rotation, attention."""

    def __init__(self, width, hq, hkv, d, capacity, batch, dtype):
        self.hq, self.hkv, self.d, self.capacity, self.batch = hq, hkv, d, capacity, batch
        self.w = _randn(width, (hq + 2 * hkv) * d, dtype=dtype, seed=1, scale=width ** -0.5)
        self.q_gain = 1 + _randn(d, dtype=dtype, seed=2, scale=0.1)
        self.k_gain = 1 + _randn(d, dtype=dtype, seed=3, scale=0.1)
        self.phases, self.m = api.rope_build_phases(d, scaling=_lib.RPE_ROPE_YARN, factor=4.0,
                                                    context=4096, low=1.0, high=32.0)
        self.k, self.v = (torch.full((batch * capacity, hkv, d), float("nan"), dtype=dtype,
                                     device="cuda") for _ in range(2))
        self.starts = _ints([b * capacity for b in range(batch + 1)])

    def project(self, x):
        return (x @ self.w).view(x.shape[0], self.hq + 2 * self.hkv, self.d)

    def step(self, x, positions, rows, cu_q, k_lens, out, workspace=None):
        """rows: where in the cache each token's key and value go."""
        qkv = self.project(x)
        q, k, v = qkv.split([self.hq, self.hkv, self.hkv], 1)
        api.qk_norm_rope_fwd(q, k, self.q_gain, self.k_gain, positions, self.phases,
                             magnitude=self.m, q_out=q, k_out=k)
        self.k.index_copy_(0, rows, k)
        self.v.index_copy_(0, rows, v)
        api.packed_attn_fwd(q, self.k, self.v, cu_q, self.starts, k_lens=k_lens, causal=True, out=out,
                            workspace=workspace)
        return q


@pytest.mark.parametrize("hq,hkv,d,dtype", [(8, 2, 128, BF16), (6, 6, 64, F16)])
def test_prompts_then_single_tokens(hq, hkv, d, dtype):
    lens, capacity, width = [130, 1, 517, 64], 600, 256
    B, total = len(lens), sum(lens)
    layer = Layer(width, hq, hkv, d, capacity, B, dtype)
    steps = 3
    x = _randn(total + steps * B, width, dtype=dtype, seed=4)
    freqs, m = _freqs(d, scaling=_lib.RPE_ROPE_YARN, factor=4.0, context=4096, low=1.0, high=32.0)
    seq = [b for b in range(B) for _ in range(lens[b])]
    pos = [i for n in lens for i in range(n)]

    def stage(x, pos, seq, cu, k_lens):
        rows = torch.tensor([b * capacity + p for b, p in zip(seq, pos)], device="cuda")
        raw = layer.project(x)
        out = torch.empty(len(pos), hq, d, dtype=dtype, device="cuda")
        q = layer.step(x, _ints(pos), rows, cu, _ints(k_lens), out)
        at = torch.tensor(pos)[:, None]
        check_rope(q, ref_rope(raw[:, :hq], at, freqs, 1, m, norm=_lib.RPE_NORM_RMS, gain=layer.q_gain))
        check_rope(layer.k[rows], ref_rope(raw[:, hq:hq + hkv], at, freqs, 1, m,
                                           norm=_lib.RPE_NORM_RMS, gain=layer.k_gain))
        assert torch.equal(layer.v[rows], raw[:, hq + hkv:])
        starts = cu.tolist()
        for b in range(B):
            mine, keys = slice(starts[b], starts[b + 1]), slice(b * capacity, b * capacity + k_lens[b])
            y, allowed, _, _ = ref_attn(q, layer.k, layer.v, mine, keys, True, d ** -0.5)
            assert bool(((out[mine].double() - y).abs() <= allowed).all()), f"sequence {b}"

    stage(x[:total], pos, seq, _cu(lens), lens)
    for t in range(steps):
        now = [n + t for n in lens]
        stage(x[total + t * B:total + (t + 1) * B], now, list(range(B)), _cu([1] * B),
              [n + 1 for n in now])


def test_a_captured_step_follows_its_inputs():
    # one captured step, replayed while positions, rows and lengths move on in place
    B, capacity, width, hq, hkv, d = 3, 2500, 128, 8, 2, 128
    lens = [7, 2300, 128]
    make = lambda: Layer(width, hq, hkv, d, capacity, B, BF16)  # noqa: E731
    eager, graphed = make(), make()
    for layer in (eager, graphed):
        for b, n in enumerate(lens):
            layer.k[b * capacity:b * capacity + n] = _randn(n, hkv, d, seed=20 + b)
            layer.v[b * capacity:b * capacity + n] = _randn(n, hkv, d, seed=30 + b)
    x, cu = _randn(B, width, seed=5), _cu([1] * B)
    pos, rows, k_lens = _ints(lens), torch.zeros(B, dtype=torch.int64, device="cuda"), _ints(lens)
    out = torch.empty(B, hq, d, dtype=BF16, device="cuda")
    size = api.packed_attn_workspace(B, B * capacity, B, hq, hkv, d)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def move(t):
        pos.copy_(_ints([n + t for n in lens]))
        k_lens.copy_(_ints([n + t + 1 for n in lens]))
        rows.copy_(torch.tensor([b * capacity + n + t for b, n in enumerate(lens)]))
        x.copy_(_randn(B, width, seed=100 + t))

    move(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # the library product's own set-up
        graphed.project(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        graphed.step(x, pos, rows, cu, k_lens, out, ws)
    for t in range(5):
        move(t)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(out)
        eager.step(x, pos, rows, cu, k_lens, want)
        assert torch.equal(out, want) and bool(torch.isfinite(out.float()).all())


def test_rotated_grid_into_the_grid_attention():
    # [B, N, heads, d] projections turned into the layout that rpe_attn_fwd reads; with tables of
    # zeros it is plain attention, which packed_attn_fwd over the same images gives too
    B, H, W, heads, d = 3, 14, 14, 6, 64
    N = H * W
    qkv = _randn(B, N, 3 * heads, d, seed=40)
    pos = torch.stack([torch.arange(N) // W, torch.arange(N) % W], 1).to(torch.int32).cuda()
    phases, _ = api.rope_build_phases(d, axes=2)
    q, k = (torch.empty(B, heads, N, d, dtype=BF16, device="cuda") for _ in range(2))
    api.qk_norm_rope_fwd(qkv[:, :, :heads], qkv[:, :, heads:2 * heads], None, None, pos, phases,
                         q_out=q.transpose(1, 2), k_out=k.transpose(1, 2))
    v = qkv[:, :, 2 * heads:].transpose(1, 2).contiguous()
    lut, _, nb = api.rpe_build_bucket_ids(H, W, *workloads.index_constants(1.9))
    zero = torch.zeros(nb, d, dtype=BF16, device="cuda")
    grid = api.rpe_attn_fwd(q, k, v, lut, nb, H, W, _lib.RPE_TERM_K, table_k=zero)
    flat = [t.transpose(1, 2).reshape(B * N, heads, d) for t in (q, k, v)]
    out, lse = api.packed_attn_fwd(*flat, _cu([N] * B), return_lse=True)
    starts = [b * N for b in range(B)]
    check_attn(*flat, [N] * B, [N] * B, starts, starts, out, lse, False, d ** -0.5)
    for b in range(B):
        y = ref_attn(*flat, slice(b * N, (b + 1) * N), slice(b * N, (b + 1) * N), False, d ** -0.5)[0]
        # 2e-2: rpe_attn_fwd's stated error in bf16
        assert float((grid[b].transpose(0, 1).double() - y).abs().max()) <= 2e-2


def test_the_quick_way_and_the_checked_way_agree(monkeypatch):
    if _lib.bind() is _lib._NoBind:
        pytest.skip("the extension module is not built")
    x = _randn(50, 8, 64, seed=50)
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    pos, (phases, _) = torch.arange(50, dtype=torch.int32, device="cuda"), api.rope_build_phases(64)
    gain = torch.linspace(0.5, 2.0, 64, device="cuda")
    cache = _randn(4000, 2, 64, seed=51)

    def calls():
        out = torch.full((50, 4, 64), 3.0, dtype=BF16, device="cuda")
        yield from api.rope_fwd(q, k, pos, phases, interleaved=True, inverse=True, magnitude=1.5)
        yield api.rope_fwd(q, None, pos[:, None], phases)[0]
        yield from api.qk_norm_rope_fwd(q, k, gain, None, pos, phases, norm=_lib.RPE_NORM_LAYER, eps=1e-3)
        yield from api.qk_norm_rope_fwd(q, k, None, gain.to(BF16))
        yield from api.packed_attn_fwd(q, k, v, _ints([3, 20, 47]), causal=True, scale=0.3, out=out,
                                       return_lse=True)
        yield api.packed_attn_fwd(q[:2], cache, cache, _cu([1, 1]), _ints([0, 2000, 4000]),
                                  k_lens=_ints([1500, 3]))

    quick = [t.clone() for t in calls()]
    monkeypatch.setattr(_lib, "_bind", _lib._NoBind)
    checked = list(calls())
    for i, (a, b) in enumerate(zip(quick, checked)):
        if i == 8:  # lse: rows of no sequence are not written
            a, b = a[3:47], b[3:47]
        assert torch.equal(a, b), f"tensor {i}"


def test_offsets_past_32_bits():
    # rows 2^30 elements apart, and a cache of more than 2^31 elements whose last rows are read
    far = 2 ** 30 + 64
    buf = torch.empty(2 * far + 4 * 64, dtype=BF16, device="cuda")
    x = torch.as_strided(buf, (3, 4, 64), (far, 64, 1))
    x.copy_(_randn(3, 4, 64, seed=60))
    near = x.contiguous()
    pos, (phases, _) = _ints([5, 6, 7]), api.rope_build_phases(64)
    want, _ = api.qk_norm_rope_fwd(near, None, None, None, pos, phases)
    want_attn = api.packed_attn_fwd(want, near, near, _cu([3]), causal=True)
    got, _ = api.qk_norm_rope_fwd(x, None, None, None, pos, phases)
    assert torch.equal(got, want)
    assert torch.equal(api.packed_attn_fwd(got, x, x, _cu([3]), causal=True), want_attn)
    api.qk_norm_rope_fwd(x, None, None, None, pos, phases, q_out=x)
    assert torch.equal(x, want)
    api.packed_attn_fwd(want, near, near, _cu([3]), causal=True, out=x)
    assert torch.equal(x, want_attn)
    del buf, x
    capacity, B, hkv, d, n = 300000, 8, 8, 128, 1000
    assert (B - 1) * capacity * hkv * d > 2 ** 31
    for nq in (1, 200):
        q = _randn(B * nq, 16, d, seed=61)
        k, v = (torch.empty(B * capacity, hkv, d, dtype=BF16, device="cuda") for _ in range(2))
        small = [_randn(B * n, hkv, d, seed=62 + i) for i in range(2)]
        for b in range(B):
            for t, s in zip((k, v), small):
                t[(b + 1) * capacity - n:(b + 1) * capacity] = s[b * n:(b + 1) * n]
        cu_q = _cu([nq] * B)
        # the sequence before ends where this one's keys begin: its own are k_lens long
        cu_k = _ints([0] + [(b + 1) * capacity - n for b in range(1, B)] + [B * capacity])
        lens = _ints([0] + [n] * (B - 1))
        got = api.packed_attn_fwd(q, k, v, cu_q, cu_k, k_lens=lens, causal=True)
        want = api.packed_attn_fwd(q, *small, cu_q, _cu([n] * B), k_lens=lens, causal=True)
        assert torch.equal(got[:nq], torch.zeros_like(got[:nq]))
        # the same keys in the same tiles, cut into pieces elsewhere at most
        starts = [b * nq for b in range(B)]
        _, lse = api.packed_attn_fwd(q, k, v, cu_q, cu_k, k_lens=lens, causal=True, return_lse=True)
        check_attn(q, *small, [nq] * (B - 1), [n] * (B - 1), starts[1:], [b * n for b in range(1, B)],
                   got, lse, True, d ** -0.5)
        check_attn(q, *small, [nq] * (B - 1), [n] * (B - 1), starts[1:], [b * n for b in range(1, B)],
                   want, lse, True, d ** -0.5)
        del k, v


@pytest.mark.parametrize("d", [8, 40, 72, 104])
@pytest.mark.parametrize("nq,nk", [([1, 1, 1], [700, 4000, 1]), ([60, 1, 130], [3000, 900, 2100])])
def test_pieces_of_any_head_size(nq, nk, d):
    _run(nq, nk, 6, 2, d, True, BF16, seed=70, capacity=4100)
    _run(nq, nk, 6, 2, d, False, F16, seed=71)


@pytest.mark.parametrize("nq,nk", [([1, 1], [3000, 50]), ([40, 100], [3000, 1500])])
def test_pieces_of_a_cache_with_heads_outside(nq, nk):
    total, d = sum(nk), 128
    q = _randn(4, sum(nq), d, seed=80).transpose(0, 1)
    k, v = (_randn(2, total, d, seed=81 + i).transpose(0, 1) for i in range(2))
    out = torch.empty(4, sum(nq), d, dtype=BF16, device="cuda").transpose(0, 1)
    out, lse = api.packed_attn_fwd(q, k, v, _cu(nq), _cu(nk), causal=True, out=out, return_lse=True)
    check_attn(q, k, v, nq, nk, _cu(nq).tolist(), _cu(nk).tolist(), out, lse, True, d ** -0.5)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("queries", [1, 90])
def test_shares_of_uneven_sequences(queries, seed):
    # one long sequence among empty, single and short ones, in any order: the CTAs' shares begin
    # and end at every place of an item, its start included
    rng = random.Random(seed)
    B = rng.choice([1, 5, 33, 70]) if queries == 1 else rng.choice([1, 2, 5])
    nk = [rng.choice([0, 1, 2, 100, 128, 129, 300]) for _ in range(B)]
    nk[rng.randrange(B)] = 512 * B + rng.randrange(9000)
    nq = [rng.randint(0 if B > 1 else 1, queries) for _ in range(B)]
    _run(nq, nk, 4, 2, 128, seed % 2 == 0, BF16, seed=90 + seed)
    _run(nq, nk, 4, 4, 64, seed % 2 == 1, F16, seed=190 + seed)


def test_growing_scores_in_every_kind_of_share():
    n, d = 4096, 128
    k = (torch.arange(n, device="cuda") / 64.0)[:, None, None].expand(n, 1, d).to(F16).contiguous()
    v = _randn(n, 1, d, dtype=F16, seed=85)
    for nq in (1, 200):
        q = torch.ones(nq, 1, d, device="cuda", dtype=F16)
        out, lse = api.packed_attn_fwd(q, k, v, _cu([nq]), _cu([n]), scale=0.5, return_lse=True)
        check_attn(q, k, v, [nq], [n], [0], [0], out, lse, False, 0.5)


@pytest.mark.parametrize("batch,tokens,hq,hk,d", [(7, 3, 2, 1, 64), (5, 1, 1, 1, 128), (2, 301, 1, 0, 64),
                                                  (3, 50, 2, 2, 40), (2, 33, 32, 8, 128)])
def test_batches_of_few_tokens_and_few_heads(batch, tokens, hq, hk, d):
    # runs of rows that cross tokens and sequences, and tokens of many heads
    x = _randn(batch, tokens, hq + hk, d, seed=95)
    pos = _ints([[[17 * b + t] for t in range(tokens)] for b in range(batch)])
    phases, _ = api.rope_build_phases(d)
    freqs, _ = _freqs(d)
    q, k = x[:, :, :hq], x[:, :, hq:] if hk else None
    for p in (pos, pos[0].contiguous()):
        outs = api.qk_norm_rope_fwd(q, k, None, None, p, phases)
        plain = api.rope_fwd(q, k, p, phases)
        at = p.cpu() if p.dim() == 3 else p.cpu()[None].expand(batch, tokens, 1)
        for src, normed, turned in zip((q, k), outs, plain):
            if src is not None:
                check_rope(normed, ref_rope(src, at, freqs, 1, norm=_lib.RPE_NORM_RMS))
                check_rope(turned, ref_rope(src, at, freqs, 1))


@pytest.mark.parametrize("causal", [False, True])
def test_no_keys_no_queries_no_sequences(causal):
    q, none = _randn(5, 4, 64, seed=97), torch.empty(0, 2, 64, dtype=BF16, device="cuda")
    out, lse = api.packed_attn_fwd(q, none, none, _cu([2, 3]), _ints([0, 0, 0]), causal=causal,
                                   return_lse=True)
    assert not bool(out.any()) and bool((lse == -float("inf")).all())
    assert api.packed_attn_fwd(q[:0], q[:, :2], q[:, :2], _cu([0]), _cu([5])).shape == (0, 4, 64)
    kept = torch.full_like(q, 2.0)
    api.packed_attn_fwd(q, q, q, _ints([0]), out=kept)
    assert bool((kept == 2).all())


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("hq,hkv,d,dtype", [(6, 3, 80, BF16), (4, 4, 64, F16), (4, 2, 128, BF16),
                                            (5, 5, 24, BF16), (8, 1, 128, F16)])
def test_short_sequences(hq, hkv, d, dtype, causal):
    # two heads of a sequence at once, an odd head left over, long sequences and empty ones among
    # them, keys of one tile and more, none at all, NaN behind the keys
    rng = random.Random(hq * d)
    tile = 128 * hkv // hq
    sizes = [0, 1, 2, tile // 3, tile // 2, tile - 1, tile]
    nq = [rng.choice(sizes) for _ in range(400)]
    nq[7], nq[300], nq[301] = tile + 1, 5 * tile + 3, 2 * tile
    _run(nq, nq, hq, hkv, d, causal, dtype, seed=200)
    nk = [rng.choice([0, 1, 40, 95, 96, 97, 128, 129, 200]) for _ in nq]
    _run(nq, nk, hq, hkv, d, causal, dtype, seed=201, capacity=210)
