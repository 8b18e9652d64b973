"""4-bit block cache and rotary positions, what needs no GPU: the layout that the header states,
the quantisation rule, and the calls that are refused before any launch."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

import trainable_sparse_attention_decode_gb300 as nosa
from oracle import quant4_oracle as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED = 1, 7


def _cfg(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype="bf16", k=1, k_e=0, max_context=64)
    base.update(kw)
    return nosa.nosa_config(**base)


@pytest.mark.parametrize("d", [64, 128])
def test_unit_layout_is_a_permutation(d):
    (kb, ks), (vb, vs) = Q.code_places(d)
    every = np.concatenate([(8 * kb + ks).ravel(), (8 * vb + vs).ravel()])
    assert np.array_equal(np.sort(every), 4 * np.arange(2 * 64 * d))
    ks, kz, vs, vz = Q.places(d)
    assert np.array_equal(np.sort(ks), 64 * d + np.arange(d))
    for at, first in ((kz, 65 * d), (vs.ravel(), 67 * d), (vz.ravel(), 69 * d)):
        assert np.array_equal(np.sort(at), first + 2 * np.arange(d))


def test_unit_bytes():
    assert nosa.nosa_quant4_unit_bytes(_cfg()) == Q.unit_bytes(128) == 9376
    assert nosa.nosa_quant4_unit_bytes(_cfg(head_dim=64)) == Q.unit_bytes(64) == 4832
    assert nosa.nosa_quant4_unit_bytes(_cfg(head_dim=96)) == 0


def test_rope_struct_matches_header(tmp_path):
    fields = [f for f, _ in nosa._Rope._fields_]
    prog = tmp_path / "rope.c"
    prog.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "nosa.h"\nint main(void) {\nprintf("%zu\\n", sizeof(nosa_rope));\n'
                    + "".join(f'printf("%zu\\n", offsetof(nosa_rope, {f}));\n' for f in fields) + "return 0;\n}\n")
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(prog), "-o", str(tmp_path / "rope")], check=True)
    got = list(map(int, subprocess.run([str(tmp_path / "rope")], capture_output=True, text=True, check=True).stdout.split()))
    assert got == [C.sizeof(nosa._Rope)] + [getattr(nosa._Rope, f).offset for f in fields]


@pytest.mark.parametrize("d", [64, 128])
def test_codes_are_within_half_a_step(d):
    """A code is the nearest one: the value is off by at most half a step, but for the roundings of the
    difference (2^-24 of it) and of 1 / step."""
    rng = np.random.default_rng(d)
    k = rng.normal(size=(3, 64, d)) + 8 * rng.normal(size=(3, 1, d)) * (np.arange(d) % 16 == 3)
    v = rng.normal(size=(3, 64, d)) * rng.lognormal(size=(3, 64, 1))
    e = rng.normal(size=(3, 64)).astype(np.float32)
    e[1, 5:9] = -np.inf
    img = Q.encode(k, v, e)
    k4, v4, e4, _, _ = Q.decode(img, d)
    (_, ks, _), (_, vs, _), s, _ = Q.parts(img, d)
    live = ~np.isneginf(e)[..., None]
    assert np.array_equal(e4, e)
    for got, x, st, sc in ((k4, k, ks, s[:, 0]), (v4, v, vs, s[:, 1])):
        tol = st * sc[:, None, None] * (0.5 + 15 * 2.0 ** -22)
        assert np.all(np.abs(got - x)[np.broadcast_to(live, x.shape)] <= np.broadcast_to(tol, x.shape)[np.broadcast_to(live, x.shape)])
    # a step is at most a fifteenth of the group's range, rounded up to three bits (keys) or eleven
    span = np.where(live, k, -np.inf).max(1) - np.where(live, k, np.inf).min(1)
    assert np.all(ks[:, 0] * s[:, 0, None] <= (span / 15 + 8 * s[:, 0, None] * 2.0 ** -11) * 1.2501)


def test_rotation_pins():
    """A quarter turn swaps, positions of 0 leave, turns add up, the backward form undoes."""
    rng = np.random.default_rng(1)
    x = rng.normal(size=(2, 5, 3, 64))
    angle = np.arange(9)[:, None] * np.array([0.3 ** i for i in range(16)])
    table = np.stack([np.cos(angle), np.sin(angle)], -1)
    one = np.ones((1, 2, 5), int)
    turn = lambda y, p, **kw: Q.rotate(y, table, p, None, False, None, **kw)  # noqa: E731
    assert np.allclose(turn(turn(x, 2 * one), 3 * one), turn(x, 5 * one), atol=1e-12)
    assert np.allclose(turn(turn(x, 7 * one), 7 * one, backward=True), x, atol=1e-12)
    assert np.array_equal(turn(x, 0 * one), x)
    quarter = np.array([[[0.0, 1.0]] * 16])
    y = Q.rotate(x, quarter, 0 * one, None, True, None)
    assert np.array_equal(y[..., 0], -x[..., 1]) and np.array_equal(y[..., 1], x[..., 0]) and np.array_equal(y[..., 32:], x[..., 32:])


P = 0x10000  # stands for an aligned device pointer: the refusals come before it is used


def _rope(**kw):
    base = dict(table=P, table_len=8, rot_dim=128, interleaved=0, n_axes=1, axes=None)
    base.update(kw)
    return C.byref(nosa._Rope(**base))


def _rotate(cfg, rope=_rope(), pos=P, n=1, q=P, qs=None, qo=P, qos=None, k=P, ks=None, ko=P, kos=None, status=None):
    return nosa.lib.nosa_rotate(C.byref(cfg) if cfg else None, rope, pos, n, q, qs, qo, qos, k, ks, ko, kos, 0, status, None)


def _append(cfg, max_blocks=4, n=1, k=P, ks=None, v=P, vs=None, e=P, n_new=None, rope=None, pos=None, units=P, n_units=8, tab=P,
            tail=P, lens=P, lens_out=P, status=None):
    return nosa.lib.nosa_quant4_append(C.byref(cfg) if cfg else None, max_blocks, n, k, ks, v, vs, e, n_new, rope, pos, units,
                                       n_units, tab, tail, lens, lens_out, status, None)


def _attend(cfg, max_blocks=4, n=1, units=P, n_units=8, tab=P, tail=P, lens=P, q=P, qs=None, q_len=None, rope=None, pos=None,
            out=2 * P, lse=None, mass=None, decay=1.0, ws=P, ws_bytes=1 << 40, status=None):
    return nosa.lib.nosa_quant4_attention(C.byref(cfg) if cfg else None, max_blocks, n, units, n_units, tab, tail, lens, q, qs,
                                          q_len, rope, pos, out, lse, mass, decay, ws, ws_bytes, status, None)


def _read(cfg, units=P, n_units=8, ids=P, n=2, k=P, v=P, e=P, status=None):
    return nosa.lib.nosa_quant4_read(C.byref(cfg) if cfg else None, units, n_units, ids, n, k, v, e, status, None)


def _st(*v):
    return (C.c_int64 * 3)(*v)


BAD_ROPES = [dict(table=None), dict(table=P + 8), dict(table_len=0), dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144),
             dict(n_axes=0), dict(n_axes=5), dict(axes=(C.c_int32 * 64)(*([0] * 63 + [1]))), dict(axes=(C.c_int32 * 64)(-1))]


@pytest.mark.parametrize("kw", BAD_ROPES)
def test_rotation_refusals(kw):
    cfg = _cfg()
    assert _rotate(cfg, rope=_rope(**kw)) == INVALID and nosa.nosa_last_error()
    assert _append(cfg, rope=_rope(**kw), pos=P) == INVALID
    assert _attend(cfg, rope=_rope(**kw), pos=P) == INVALID


@pytest.mark.parametrize("kw", [
    dict(cfg=None), dict(rope=None), dict(pos=None), dict(pos=P + 2), dict(n=-1), dict(q=None), dict(qo=None), dict(k=None), dict(ko=None),
    dict(q=P + 8), dict(ko=P + 4), dict(status=P + 1), dict(qs=_st(8, 8, 4)), dict(qs=_st(-8, 8, 8)), dict(kos=_st(256, 256, 0)),
    dict(qs=_st(2048, 1024, 128))])
def test_rotate_refusals(kw):
    kw = dict(kw)
    cfg = kw.pop("cfg", _cfg())
    assert _rotate(cfg, **kw) == INVALID and nosa.nosa_last_error()


def test_rotate_in_place_wants_the_same_strides():
    assert _rotate(_cfg(), qos=_st(4096, 2048, 128)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(cfg=None), dict(max_blocks=0), dict(n=-1), dict(k=None), dict(v=None), dict(units=None), dict(n_units=-1), dict(tab=None),
    dict(tail=None), dict(lens=None), dict(lens_out=None), dict(k=P + 8), dict(units=P + 4), dict(e=P + 2), dict(ks=_st(8, 8, 4)),
    dict(vs=_st(-8, 8, 8)), dict(rope=_rope(), pos=None)])
def test_append_refusals(kw):
    kw = dict(kw)
    cfg = kw.pop("cfg", _cfg())
    assert _append(cfg, **kw) == INVALID and nosa.nosa_last_error()


@pytest.mark.parametrize("kw", [
    dict(cfg=None), dict(max_blocks=0), dict(n=0), dict(units=None), dict(tab=None), dict(tail=None), dict(lens=None), dict(q=None),
    dict(out=None), dict(ws=None), dict(out=P), dict(ws=P + 16), dict(mass=P, decay=1.5), dict(mass=P, decay=float("nan")),
    dict(qs=_st(8, 8, 4)), dict(rope=_rope(), pos=None), dict(ws_bytes=16, mass=P)])
def test_attention_refusals(kw):
    kw = dict(kw)
    cfg = kw.pop("cfg", _cfg())
    assert _attend(cfg, **kw) == INVALID and nosa.nosa_last_error()


def test_sizes_outside_the_kernels():
    cfg = _cfg()
    assert _attend(cfg, n=129) == UNSUPPORTED and _attend(cfg, max_blocks=16385) == UNSUPPORTED
    assert _append(cfg, max_blocks=16385) == UNSUPPORTED
    assert nosa.nosa_quant4_attention_workspace_bytes(cfg, 4, 129) == 0
    assert nosa.nosa_quant4_attention_workspace_bytes(cfg, 0) == 0
    assert nosa.nosa_quant4_attention_workspace_bytes(cfg, 4) > 0


@pytest.mark.parametrize("kw", [dict(cfg=None), dict(n=-1), dict(n_units=-1), dict(units=None), dict(units=P + 8), dict(k=P + 8),
                                dict(e=P + 2), dict(ids=P + 1), dict(ids=None, n=9)])
def test_read_refusals(kw):
    kw = dict(kw)
    cfg = kw.pop("cfg", _cfg())
    assert _read(cfg, **kw) == INVALID and nosa.nosa_last_error()


def test_binding_refusals_without_a_gpu():
    cfg = _cfg()
    t = torch.zeros(4, 64, 2)
    for bad in (t, t[..., 0], 5, None):
        with pytest.raises(ValueError):
            nosa.nosa_rope(bad)
    with pytest.raises(ValueError):
        nosa.nosa_rotate(cfg, None, None, torch.zeros(2, 1, 8, 128))
    with pytest.raises(ValueError):
        nosa.nosa_rotate(cfg, object(), None, torch.zeros(2, 1, 8, 128))
    with pytest.raises(ValueError):
        nosa.nosa_quant4_read(cfg, torch.zeros(9376, dtype=torch.uint8))
    with pytest.raises(ValueError):
        nosa.nosa_quant4_read(cfg, None, torch.zeros(1, 64, 128))
    with pytest.raises(ValueError):
        nosa.nosa_quant4_append(cfg, None, None, None, None, None, None, None)
    with pytest.raises(ValueError):
        nosa.nosa_quant4_attention(cfg, None, None, None, None, None, None)
