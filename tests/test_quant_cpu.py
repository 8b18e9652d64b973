"""8-bit block cache, what needs no GPU: the layout that the header states, the
oracle's number format, and the calls that are refused before any launch."""
import ctypes as C

import numpy as np
import pytest
import torch

import trainable_sparse_attention_decode_gb300 as nosa
from oracle import quant_oracle as Q

OK, INVALID, UNSUPPORTED = 0, 1, 7


def _cfg(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, dtype="bf16", k=1, k_e=0, max_context=64)
    base.update(kw)
    return nosa.nosa_config(**base)


@pytest.mark.parametrize("d", [64, 128])
def test_unit_layout_is_a_permutation(d):
    k, v = Q.code_offsets(d)
    every = np.concatenate([k.ravel(), v.ravel()])
    assert np.array_equal(np.sort(every), np.arange(2 * 64 * d))
    # a slice of 16 tokens is one run: its key codes, then its value codes
    for w in range(4):
        t = slice(16 * w, 16 * w + 16)
        assert k[t].min() == 32 * d * w and k[t].max() == 32 * d * w + 16 * d - 1
        assert v[t].min() == 32 * d * w + 16 * d and v[t].max() == 32 * d * (w + 1) - 1


def test_unit_bytes():
    assert nosa.nosa_quant_unit_bytes(_cfg()) == Q.unit_bytes(128) == 16672
    assert nosa.nosa_quant_unit_bytes(_cfg(head_dim=64)) == Q.unit_bytes(64) == 8480
    assert nosa.nosa_quant_unit_bytes(_cfg(head_dim=96)) == 0


def test_oracle_numbers_are_e4m3():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(np.isnan(t), np.isnan(Q.E4M3))
    assert np.array_equal(t[~np.isnan(t)], Q.E4M3[~np.isnan(t)])
    x = np.random.default_rng(0).normal(size=(3, 64, 64)) * 3
    e = np.zeros((3, 64))
    k8, _, _, s = Q.decode(Q.encode(x, x, e), 64)
    y = x / s[:, 0, None, None]
    assert np.all(np.abs(k8 - y) <= Q.nearest_distance(y) * (1 + 1e-12))
    # a rounding is off by at most half a step: 2^-4 of the value, or half the smallest number
    assert np.all(np.abs(k8 - y) <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10))


P = 0x10000  # stands for an aligned device pointer: the refusals come before it is used


def _append(cfg, max_blocks=4, n=1, k=P, ks=None, v=P, vs=None, e=P, n_new=None, units=P, n_units=8, tab=P, tail=P,
            lens=P, lens_out=P, status=None):
    return nosa.lib.nosa_quant_append(C.byref(cfg) if cfg else None, max_blocks, n, k, ks, v, vs, e, n_new, units,
                                      n_units, tab, tail, lens, lens_out, status, None)


def _attention(cfg, max_blocks=4, n=1, units=P, n_units=8, tab=P, tail=P, lens=P, q=P, qs=None, q_len=None, out=2 * P,
               lse=None, mass=None, decay=1.0, ws=P, ws_bytes=1 << 40, status=None):
    return nosa.lib.nosa_quant_attention(C.byref(cfg) if cfg else None, max_blocks, n, units, n_units, tab, tail, lens,
                                         q, qs, q_len, out, lse, mass, decay, ws, ws_bytes, status, None)


def _evict(cfg, max_blocks=4, budget=2, recent=1, tab=P, mass=P, lens=P, tab_out=P, mass_out=P, lens_out=P, order=None,
           status=None):
    return nosa.lib.nosa_quant_evict(C.byref(cfg) if cfg else None, max_blocks, budget, recent, tab, mass, lens, tab_out,
                                     mass_out, lens_out, order, status, None)


@pytest.mark.parametrize("kw,status", [
    (dict(max_blocks=0), INVALID), (dict(max_blocks=16385), UNSUPPORTED), (dict(n=-1), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(units=None), INVALID), (dict(n_units=-1), INVALID), (dict(tab=None), INVALID),
    (dict(tail=None), INVALID), (dict(lens=None), INVALID), (dict(lens_out=None), INVALID), (dict(k=P + 8), INVALID),
    (dict(v=P + 4), INVALID), (dict(units=P + 8), INVALID), (dict(tail=P + 8), INVALID), (dict(e=P + 2), INVALID),
    (dict(n_new=P + 1), INVALID), (dict(lens=P + 2), INVALID), (dict(status=P + 2), INVALID),
    (dict(ks=(C.c_int64 * 3)(1024, 4, 128)), INVALID), (dict(vs=(C.c_int64 * 3)(-1024, 256, 128)), INVALID)])
def test_append_refusals(kw, status):
    assert _append(_cfg(), **kw) == status
    assert nosa.nosa_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(max_blocks=0), INVALID), (dict(max_blocks=16385), UNSUPPORTED), (dict(n=0), INVALID),
    (dict(n=129), UNSUPPORTED), (dict(units=None), INVALID), (dict(tab=None), INVALID), (dict(tail=None), INVALID),
    (dict(lens=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ws=None), INVALID),
    (dict(ws=P + 16), INVALID), (dict(q=P + 8), INVALID), (dict(out=P + 8), INVALID), (dict(lse=P + 2), INVALID),
    (dict(mass=P + 1), INVALID), (dict(mass=P, decay=1.5), INVALID), (dict(mass=P, decay=-0.1), INVALID),
    (dict(mass=P, decay=float("nan")), INVALID), (dict(out=P), INVALID), (dict(qs=(C.c_int64 * 3)(1024, 1024, 4)), INVALID)])
def test_attention_refusals(kw, status):
    assert _attention(_cfg(), **kw) == status
    assert nosa.nosa_last_error() != ""


@pytest.mark.parametrize("kw,status", [
    (dict(max_blocks=0), INVALID), (dict(max_blocks=16385), UNSUPPORTED), (dict(budget=0), INVALID),
    (dict(recent=-1), INVALID), (dict(recent=3), INVALID), (dict(tab=None), INVALID), (dict(mass=None), INVALID),
    (dict(lens=None), INVALID), (dict(tab_out=None), INVALID), (dict(mass_out=None), INVALID),
    (dict(lens_out=None), INVALID), (dict(order=P + 2), INVALID), (dict(mass=P + 1), INVALID)])
def test_evict_refusals(kw, status):
    assert _evict(_cfg(), **kw) == status
    assert nosa.nosa_last_error() != ""


@pytest.mark.parametrize("call", [_append, _attention, _evict])
@pytest.mark.parametrize("bad,status", [(None, INVALID), (dict(n_q_heads=7), INVALID), (dict(n_q_heads=10), UNSUPPORTED),
                                        (dict(head_dim=96), UNSUPPORTED)])
def test_bad_configurations_are_refused(call, bad, status):
    assert call(None if bad is None else _cfg(**bad)) == status


def test_workspace_query_refuses():
    f = nosa.nosa_quant_attention_workspace_bytes
    assert f(_cfg(head_dim=96), 4) == 0 and f(_cfg(), 0) == 0 and f(_cfg(), 16385) == 0
    assert f(_cfg(), 4, 0) == 0 and f(_cfg(), 4, 129) == 0


def test_binding_refuses_cpu_tensors():
    cfg = _cfg()
    z = torch.zeros
    U = 4
    k = z(2, 1, 2, 128, dtype=torch.bfloat16)
    units, tab = z(8, 16672, dtype=torch.uint8), z(U, 4, dtype=torch.int32)
    tail, lens = z(U, nosa.nosa_payload_bytes(cfg), dtype=torch.uint8), z(U, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        nosa.nosa_quant_append(cfg, k, k, None, units, tab, tail, lens)
    with pytest.raises(ValueError, match="CUDA"):
        nosa.nosa_quant_evict(cfg, 2, 1, tab, z(U, 4), lens)
    q = z(2, 1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        nosa.nosa_quant_attention(cfg, units, tab, tail, lens, q, torch.empty_like(q))


# ---- the oracle's own eviction against enumeration -----------------------------------------------------------------
def test_oracle_evict_keeps_the_heaviest():
    import itertools
    rng = np.random.default_rng(3)
    for _ in range(200):
        full, cap = int(rng.integers(1, 8)), 9
        budget = int(rng.integers(1, 9))
        recent = int(rng.integers(0, budget + 1))
        mass = rng.integers(0, 3, size=cap).astype(np.float32)
        tab = rng.permutation(cap)
        t, m, n, order = Q.evict(tab, mass, 64 * full + 7, budget, recent)
        keep = min(full, budget)
        assert n == 64 * keep + 7 and sorted(order) == list(range(cap))
        assert np.array_equal(t, tab[order]) and list(order[:keep]) == sorted(order[:keep])
        if full <= budget:
            assert np.array_equal(m, mass)
            continue
        best = max((sum(mass[list(c)]) for c in itertools.combinations(range(full - recent), keep - recent)))
        assert sum(mass[order[:keep - recent]]) == best
        assert list(order[keep - recent:keep]) == list(range(full - recent, full))
        assert m[keep] == mass[full] and not m[keep + 1:full + 1].any()


@pytest.mark.parametrize("bad", [None, 4096, np.zeros((2, 1, 2, 128), np.float32), [1, 2], "x"])
def test_binding_refuses_what_is_no_tensor(bad):
    """A tensor that is missing, and pointers, arrays and lists in its place: a ValueError."""
    cfg, U, z = _cfg(), 4, torch.zeros
    k, q = z(2, 1, 2, 128, dtype=torch.bfloat16), z(2, 1, 8, 128, dtype=torch.bfloat16)
    cache = dict(units=z(8, 16672, dtype=torch.uint8), block_tab=z(U, 4, dtype=torch.int32),
                 tail=z(U, nosa.nosa_payload_bytes(cfg), dtype=torch.uint8), lens=z(U, dtype=torch.int32))
    calls = [(nosa.nosa_quant_append, dict(k=k, v=k, **cache), dict(e=None)),
             (nosa.nosa_quant_attention, dict(q=q, out=torch.empty_like(q), **cache), {}),
             (nosa.nosa_quant_evict, dict(block_tab=cache["block_tab"], mass=z(U, 4), lens=cache["lens"]),
              dict(budget=2, n_recent=1))]
    for f, tensors, others in calls:
        for name in tensors:
            with pytest.raises(ValueError):  # (or the tensors before it are, which are the CPU's)
                f(cfg, **{**tensors, name: bad}, **others)
    if bad is not None:
        with pytest.raises(ValueError):
            nosa.nosa_quant_append(cfg, **calls[0][1], e=bad)


def test_binding_refuses_tensors_of_other_ranks():
    cfg, U, z = _cfg(), 4, torch.zeros
    with pytest.raises(ValueError, match="block_tab"):
        nosa.nosa_quant_evict(cfg, 2, 1, z(U, dtype=torch.int32), z(U, 4), z(U, dtype=torch.int32))
    q = z(8, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must have 4"):
        nosa.nosa_quant_attention(cfg, z(8), z(U, 4, dtype=torch.int32), z(8), z(U), q, q)
