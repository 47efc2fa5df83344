"""Refusals of the calls on tokens (rotary positions, norms, packed attention), made on
the host before any launch, so no GPU is needed."""
import ctypes

import pytest

from vision_transformer_attention_gb300 import _lib

OK, INVALID, UNSUPPORTED = _lib.RPE_OK, _lib.RPE_ERR_INVALID_ARG, _lib.RPE_ERR_UNSUPPORTED
FAKE = 1 << 20


def _view(ptr=FAKE, b=0, t=256, h=64):
    return ctypes.byref(_lib.View(ptr, b, t, h))


ROPE = dict(q=None, k=None, q_out=None, k_out=None, positions=FAKE, axes=1, phases=FAKE, rd=64,
            magnitude=1.0, flags=0, batch=1, tokens=8, hq=4, hk=2, d=64, dtype=0, stream=None)


def _rope(**kw):
    a = dict(ROPE, q=_view(), k=_view(), q_out=_view(), k_out=_view())
    a.update(kw)
    return _lib.lib().rope_fwd(*a.values())


def _norm(norm=0, eps=1e-6, gain_q=None, gain_k=None, gain_dtype=1, **kw):
    a = dict(ROPE, q=_view(), k=_view(), q_out=_view(), k_out=_view())
    a.update(kw)
    v = list(a.values())
    return _lib.lib().qk_norm_rope_fwd(*v[:4], norm, eps, gain_q, gain_k, gain_dtype, *v[4:])


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(q_out=None)),
    (INVALID, dict(q=_view(0))), (INVALID, dict(q=_view(FAKE + 1))),
    (INVALID, dict(dtype=1, q=_view(FAKE + 2))), (INVALID, dict(q=_view(t=-1))),
    (INVALID, dict(q_out=_view(t=0))), (INVALID, dict(k_out=_view(h=0))),
    (INVALID, dict(batch=2, q_out=_view(b=0))), (INVALID, dict(batch=-1)),
    (INVALID, dict(tokens=-1)), (INVALID, dict(hq=0)), (INVALID, dict(hk=-1)),
    (INVALID, dict(d=0)), (INVALID, dict(rd=66)), (INVALID, dict(rd=63)), (INVALID, dict(rd=0)),
    (INVALID, dict(rd=62, axes=2)), (INVALID, dict(axes=3)), (INVALID, dict(axes=0)),
    (INVALID, dict(flags=8)), (INVALID, dict(dtype=3)), (INVALID, dict(magnitude=float("nan"))),
    (INVALID, dict(positions=None)), (INVALID, dict(phases=None)),
    (INVALID, dict(phases=FAKE + 4)), (UNSUPPORTED, dict(d=264)),
    (UNSUPPORTED, dict(hq=65537)), (UNSUPPORTED, dict(batch=1 << 16, tokens=1 << 16)),
    (OK, dict(tokens=0, q=None, k=None)), (OK, dict(batch=0))])
def test_rope_refusals(want, kw):
    assert _rope(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(norm=2)), (INVALID, dict(eps=-1.0)), (INVALID, dict(eps=float("inf"))),
    (INVALID, dict(gain_dtype=2)), (INVALID, dict(gain_q=FAKE + 2)),
    (INVALID, dict(flags=_lib.RPE_ROPE_INVERSE)), (INVALID, dict(k=None)),
    (INVALID, dict(positions=None)), (UNSUPPORTED, dict(d=257)),
    (OK, dict(tokens=0, rd=0, positions=None, phases=None))])
def test_norm_refusals(want, kw):
    assert _norm(**kw) == want


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(phases=None)), (INVALID, dict(phases=FAKE + 4)), (INVALID, dict(rd=0)),
    (INVALID, dict(rd=7)), (INVALID, dict(rd=6, axes=2)), (INVALID, dict(axes=4)),
    (INVALID, dict(scaling=5)), (INVALID, dict(scaling=-1)), (INVALID, dict(base=1.0)),
    (INVALID, dict(base=float("nan"))), (INVALID, dict(scaling=1, factor=0.5)),
    (INVALID, dict(scaling=2, rd=2)), (INVALID, dict(scaling=3, context=0.0)),
    (INVALID, dict(scaling=4, low=4.0, high=4.0)), (INVALID, dict(scaling=4, low=0.0)),
    (UNSUPPORTED, dict(rd=258))])
def test_phase_table_refusals(want, kw):
    a = dict(rd=64, axes=1, scaling=0, base=1e4, factor=2.0, context=4096.0, low=1.0, high=32.0,
             phases=FAKE)
    a.update(kw)
    m = ctypes.c_float(0)
    assert _lib.lib().rope_build_phases(*a.values(), ctypes.byref(m), None) == want


def _attn(**kw):
    a = dict(q=_view(), k=_view(), v=_view(), out=_view(), lse=None, cu_q=FAKE, cu_k=FAKE,
             k_lens=None, batch=2, total_q=64, total_k=64, hq=4, hkv=2, d=64, scale=0.125, flags=0,
             dtype=0, workspace=None, bytes=0, stream=None)
    a.update(kw)
    return _lib.lib().packed_attn_fwd(*a.values())


@pytest.mark.parametrize("want,kw", [
    (INVALID, dict(q=None)), (INVALID, dict(k=None)), (INVALID, dict(v=_view(0))),
    (INVALID, dict(out=None)), (INVALID, dict(q=_view(FAKE + 8))), (INVALID, dict(v=_view(t=4))),
    (INVALID, dict(k=_view(h=12))), (INVALID, dict(k=_view(h=0))), (INVALID, dict(out=_view(t=0))),
    (INVALID, dict(out=_view(t=-256))), (INVALID, dict(cu_q=None)), (INVALID, dict(cu_k=None)),
    (INVALID, dict(cu_q=FAKE + 2)), (INVALID, dict(k_lens=FAKE + 1)), (INVALID, dict(lse=FAKE + 2)),
    (INVALID, dict(batch=-1)), (INVALID, dict(total_q=-1)), (INVALID, dict(total_k=-1)),
    (INVALID, dict(hq=0)), (INVALID, dict(hkv=0)), (INVALID, dict(hq=5)), (INVALID, dict(d=0)),
    (INVALID, dict(scale=0.0)), (INVALID, dict(scale=-1.0)), (INVALID, dict(scale=float("nan"))),
    (INVALID, dict(flags=2)), (INVALID, dict(dtype=3)), (UNSUPPORTED, dict(dtype=1)),
    (UNSUPPORTED, dict(d=136)), (UNSUPPORTED, dict(d=36)), (UNSUPPORTED, dict(hq=258)),
    (UNSUPPORTED, dict(total_q=1 << 30)), (UNSUPPORTED, dict(total_k=1 << 30)),
    (UNSUPPORTED, dict(batch=1 << 24)),
    # one token against 4096 keys runs in pieces and needs its workspace
    (INVALID, dict(batch=1, total_q=1, total_k=4096)),
    (INVALID, dict(batch=1, total_q=1, total_k=4096, workspace=FAKE, bytes=64)),
    (OK, dict(total_q=0, q=None)), (OK, dict(batch=0))])
def test_packed_attention_refusals(want, kw):
    assert _attn(**kw) == want


def test_packed_attention_workspace_sizes():
    size = ctypes.c_size_t(7)
    call = lambda *a: _lib.lib().packed_attn_workspace(*a, ctypes.byref(size))  # noqa: E731
    assert call(4096, 4096, 4, 8, 2, 64, 0) == OK and size.value == 0
    assert call(1, 4096, 1, 8, 2, 64, 0) == OK and size.value > 0
    assert call(0, 4096, 1, 8, 2, 64, 0) == OK and size.value == 0
    assert call(1, 4096, 1, 8, 3, 64, 0) == INVALID
    assert call(1, 4096, 1, 8, 2, 64, 1) == UNSUPPORTED
    assert _lib.lib().packed_attn_workspace(1, 1, 1, 1, 1, 64, 0, None) == INVALID
