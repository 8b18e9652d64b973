"""Rotary positions and the 4-bit block cache on the GPU against the oracle: rotation, append,
reading back, attention, and a generation loop of them.

Tolerances. The rotation and the append are defined down to their roundings and compared bit
for bit. A value that is read back is step * n + zero in one rounding to fp32 (2^-24 of the
larger of the two, at most step * n + |zero|) and one to the type (half a step: 2^-24 or 2^-8).
Attention: with S the largest sum |q_x| (step n + |zero|)_x / sqrt(d) of a row, a logit is off
by at most 2^-18 S + 2^-22 |l|: the tensor cores add the d products of the codes and the d of
the zeros in at most d / 4 = 32 steps of truncating fp32 additions (2^-23 each, of partial sums
that S bounds), the operands of an fp32 query carry 22 bits, the scaling adds three roundings;
weights are then off by twice that relatively, plus 2^-20 for exp and normalisation and 2^-23
for each of the n / 16 additions. The weights enter the product with the zeros rounded once and
the one with the codes rounded twice (as weights and times the step), to 11 bits where the
output is bf16, to 22 where it is fp32: at most 2 * 2^-11 (2 * 2^-21) of A, the weighted mean of
step n + |zero|; the product's own additions of n terms are 2^-23 of A each 16. The output's
rounding is half a step, 2^-8 (bf16) or 2^-24 (fp32).
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import trainable_sparse_attention_decode_gb300 as nosa
from oracle import quant4_oracle as Q
from oracle.quant_oracle import evict as evict_oracle
from test_quant_gpu import B, DT, Model, config, dev, f64, make_tail, query, tail_arrays

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def rounder(dtype):
    """fp32 arrays rounded to the type, as fp64."""
    return lambda x: torch.as_tensor(np.ascontiguousarray(x, np.float32)).to(DT[dtype]).double().numpy()


class Turn:
    """A rotation: the framework's handle and the oracle's arrays."""

    def __init__(self, rot, length, axes=None, interleaved=False, base=1e4, scale=1.0):
        a = np.arange(length)[:, None] * base ** (-np.arange(rot // 2) / (rot // 2))
        self.table = (np.stack([np.cos(a), np.sin(a)], -1) * scale).astype(np.float32)
        self.axes, self.interleaved, self.n_axes = axes, interleaved, 1 if axes is None else max(axes) + 1
        self.rope = nosa.nosa_rope(dev(self.table), axes=axes, interleaved=interleaved)

    def positions(self, rng, batch, n):
        return rng.integers(0, len(self.table), size=(self.n_axes, batch, n)).astype(np.int32)

    def oracle(self, x, pos, dtype, backward=False):
        return Q.rotate(x, self.table, pos, self.axes, self.interleaved, rounder(dtype), backward)


def some_axes(kind, pairs):
    return {"one": None, "sections": [0] * (pairs // 4) + [1] * (3 * pairs // 8) + [2] * (pairs - pairs // 4 - 3 * pairs // 8),
            "uneven": [0] * (pairs // 4 + 3) + [1] * (pairs // 4 + 2) + [2] * (pairs // 2 - 5), "mixed": [i % 3 for i in range(pairs)],
            "four": [i % 4 for i in range(pairs)]}[kind]


# ---------------------------------------------------------------------------
# rotation
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("batch,n,hq,hkv,d,rot,kind,interleaved", [
    (1, 1, 1, 1, 64, 64, "one", False), (32, 1, 32, 8, 128, 128, "one", False), (2, 37, 12, 2, 128, 128, "sections", False),
    (3, 5, 6, 2, 64, 32, "uneven", True), (2, 129, 4, 4, 128, 96, "mixed", False), (1, 300, 8, 1, 64, 16, "one", True),
    (2, 3, 3, 3, 128, 112, "four", True), (1, 1000, 2, 2, 64, 48, "mixed", False), (5, 211, 8, 8, 128, 64, "uneven", False)])
def test_rotate_matches_oracle(dtype, batch, n, hq, hkv, d, rot, kind, interleaved):
    rng = np.random.default_rng(n + rot)
    turn = Turn(rot, 1777, some_axes(kind, rot // 2), interleaved)
    cfg = config(batch, hq, hkv, d, dtype)
    pos = turn.positions(rng, batch, n)
    q, k = query(rng, batch, n, hq, d, dtype, 3.0), query(rng, batch, n, hkv, d, dtype, 3.0)
    qo, ko = torch.full_like(q, 7.0), torch.full_like(k, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for backward in (False, True):
        nosa.nosa_rotate(cfg, turn.rope, dev(pos), q, k, q_out=qo, k_out=ko, backward=backward, status=status)
        want_q, want_k = turn.oracle(f64(q), pos, dtype, backward), turn.oracle(f64(k), pos, dtype, backward)
        assert np.array_equal(f64(qo), want_q) and np.array_equal(f64(ko), want_k)
    # in place, in strided rows of one array, one of the two alone
    wide = torch.randn(batch, n, hq + 2 * hkv, d, device="cuda").to(DT[dtype])
    ref = wide.clone()
    nosa.nosa_rotate(cfg, turn.rope, dev(pos), wide[:, :, :hq], wide[:, :, hq:hq + hkv], status=status)
    assert np.array_equal(f64(wide[:, :, :hq]), turn.oracle(f64(ref[:, :, :hq]), pos, dtype))
    assert np.array_equal(f64(wide[:, :, hq:hq + hkv]), turn.oracle(f64(ref[:, :, hq:hq + hkv]), pos, dtype))
    assert torch.equal(wide[:, :, hq + hkv:], ref[:, :, hq + hkv:])
    nosa.nosa_rotate(cfg, turn.rope, dev(pos), None, wide[:, :, hq + hkv:], status=status)
    assert np.array_equal(f64(wide[:, :, hq + hkv:]), turn.oracle(f64(ref[:, :, hq + hkv:]), pos, dtype))
    only = torch.empty_like(q)
    nosa.nosa_rotate(cfg, turn.rope, dev(pos), q, q_out=only)
    assert np.array_equal(f64(only), turn.oracle(f64(q), pos, dtype))
    # rows apart from each other on the way out: strided outputs
    apart = torch.zeros(n, batch, hq, 2, d, dtype=DT[dtype], device="cuda")
    nosa.nosa_rotate(cfg, turn.rope, dev(pos), q, q_out=apart[:, :, :, 1].transpose(0, 1))
    assert torch.equal(apart[:, :, :, 1].transpose(0, 1), only) and not apart[:, :, :, 0].any()
    assert status.item() == 0


@pytest.mark.parametrize("kind,interleaved", [("one", False), ("mixed", True)])
def test_rotate_gradient(kind, interleaved):
    """The backward form against the formula's transpose and against differences. The map is linear, so a
    difference quotient has only its roundings: two fp32 outputs of size <= 8 a step of 1 apart, three
    roundings of 2^-24 each, weighted by |g| and added over the row's elements."""
    rng = np.random.default_rng(3)
    batch, n, hq, d, rot = 2, 7, 2, 64, 48
    turn = Turn(rot, 90, some_axes(kind, rot // 2), interleaved, scale=1.25)  # (not a pure rotation: the transpose, not the inverse)
    cfg = config(batch, hq, hq, d, "f32")
    pos = dev(turn.positions(rng, batch, n))
    x, g = query(rng, batch, n, hq, d, "f32"), query(rng, batch, n, hq, d, "f32")
    grad = torch.empty_like(g)
    nosa.nosa_rotate(cfg, turn.rope, pos, g, q_out=grad, backward=True)
    f = lambda y: (lambda o: (nosa.nosa_rotate(cfg, turn.rope, pos, y, q_out=o), o)[1])(torch.empty_like(y))  # noqa: E731
    base = f(x).double()
    for i in range(d):
        step = x.clone()
        step[..., i] += 1.0
        moved = (step[..., i] - x[..., i]).double()  # (1 up to a rounding)
        diff = ((f(step).double() - base) * g.double()).sum(-1) / moved
        bound = (g.abs().double().sum(-1) * 1.25 * 2 * (x.abs().amax(-1).double() + 1) * 3 * 2.0 ** -24 * 2)
        assert ((diff - grad[..., i].double()).abs() <= bound + 1e-12).all()


def test_rotate_positions_out_of_range_and_far():
    rng = np.random.default_rng(5)
    turn = Turn(64, 1 << 20)
    cfg = config(1, 2, 2, 64, "bf16")
    pos = np.array([[[0, (1 << 20) - 1, 524289, -1, 1 << 20, 2 ** 31 - 1]]], np.int32)
    q = query(rng, 1, 6, 2, 64, "bf16")
    out, status = torch.empty_like(q), torch.zeros(1, dtype=torch.int32, device="cuda")
    nosa.nosa_rotate(cfg, turn.rope, dev(pos[0, :, :3].reshape(1, 1, 3)), q[:, :3].contiguous(), q_out=out[:, :3].contiguous(), status=status)
    assert status.item() == 0
    nosa.nosa_rotate(cfg, turn.rope, dev(pos[0]), q, q_out=out, status=status)
    assert status.item() == nosa.NOSA_QUANT_INDEX
    assert np.array_equal(f64(out), turn.oracle(f64(q), pos, "bf16"))  # (clamped)


def test_rotate_nothing():
    turn = Turn(64, 4)
    q = torch.zeros(2, 0, 4, 64, device="cuda")
    nosa.nosa_rotate(config(2, 4, 2, 64, "f32"), turn.rope, torch.zeros(1, 2, 0, dtype=torch.int32, device="cuda"), q, q[:, :, :2])


def test_rotate_many_rows():
    """More elements than 2^31: the last rows are turned as the first."""
    turn = Turn(128, 50)
    cfg = config(1, 8, 8, 128, "bf16")
    n = (1 << 21) + 3
    q = torch.zeros(1, n, 8, 128, dtype=torch.bfloat16, device="cuda")
    q[0, -2:] = 1.5
    q[0, :2] = 1.5
    pos = (torch.arange(n, device="cuda") % 50).to(torch.int32)[None]
    pos[0, -2:], pos[0, :2] = 7, 7
    nosa.nosa_rotate(cfg, turn.rope, pos, q)
    want = turn.oracle(np.full((1, 1, 8, 128), 1.5), np.array([[[7]]]), "bf16")[0, 0]
    for i in (0, 1, n - 2, n - 1):
        assert np.array_equal(f64(q[0, i]), want)
    assert not q[0, 2:-2].any()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,batch,hq,hkv,d,steps,strided,turned", [
    ("bf16", 2, 8, 2, 128, [1, 62, 1, 1, 64, 130, 3, 1], False, ("one", 128, False)),
    ("f32", 1, 4, 1, 64, [63, 1, 65, 200, 1], False, None),
    ("bf16", 3, 3, 3, 64, [1000, 1, 24, 64], True, ("sections", 64, False)),
    ("f32", 2, 6, 3, 128, [64, 127, 2, 1, 129], True, ("mixed", 96, True)),
    ("bf16", 1, 8, 1, 128, [1] * 66, False, ("uneven", 64, False)), ("bf16", 2, 2, 2, 128, [300, 17], False, None),
    ("f32", 3, 2, 1, 64, [70, 1, 130], False, ("four", 32, False)), ("bf16", 1, 2, 2, 64, [5, 333], True, ("one", 16, True))])
def test_append_matches_oracle(dtype, batch, hq, hkv, d, steps, strided, turned):
    rng = np.random.default_rng(sum(steps) + d)
    U, cap = batch * hkv, sum(steps) // B + 2
    cfg = config(batch, hq, hkv, d, dtype)
    turn = turned and Turn(turned[1], 700, some_axes(turned[0], turned[1] // 2), turned[2])
    extra = 3
    tab = rng.permutation(U * cap + extra)[:U * cap].reshape(U, cap).astype(np.int32)
    units = torch.full((U * cap + extra, Q.unit_bytes(d)), 0xA5, dtype=torch.uint8, device="cuda")
    tail = torch.full((U * nosa.nosa_payload_bytes(cfg),), 0x5A, dtype=torch.uint8, device="cuda")
    lens = torch.zeros(U, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    model = Model(U, d)
    t_tab = dev(tab)
    for i, n in enumerate(steps):
        wide = torch.randn(batch, n, 2 * hkv + 1, d, device="cuda").mul_(rng.uniform(0.1, 30))
        wide[:, :, :hkv] += torch.randn(hkv, d, device="cuda") * 20
        wide = wide.to(DT[dtype])
        k, v = wide[:, :, :hkv], wide[:, :, hkv:2 * hkv]
        if not strided:
            k, v = k.contiguous(), v.contiguous()
        e = rng.normal(size=(batch, n, hkv)).astype(np.float32)
        e[rng.random(size=e.shape) < 0.05] = -np.inf
        if i == 1:
            e[:] = 0.0
        n_new = rng.integers(0, n + 1, size=batch).astype(np.int32) if i % 3 == 2 else None
        pos = turn and turn.positions(rng, batch, n)
        if turn and n_new is not None:  # positions behind the valid tokens are not read
            for b in range(batch):
                pos[:, b, n_new[b]:] = -5
        before = tail.clone()
        nosa.nosa_quant4_append(cfg, k, v, None if i == 1 else dev(e), units, t_tab, tail, lens,
                                n_new=None if n_new is None else dev(n_new), rope=turn and turn.rope,
                                positions=None if turn is None else dev(pos), status=status)
        kf, vf = f64(k), f64(v)
        if turn:
            kf = turn.oracle(kf, pos, dtype)
        for u in range(U):
            b, h = divmod(u, hkv)
            m = n if n_new is None else n_new[b]
            model.add(u, kf[b, :m, h], vf[b, :m, h], e[b, :m, h].astype(np.float64))
        assert lens.tolist() == [len(x) for x in model.e]
        tk, tv, te = tail_arrays(cfg, tail, d, dtype)
        bk, bv, be = tail_arrays(cfg, before, d, dtype)
        for u in range(U):
            nf, nt = divmod(len(model.e[u]), B)
            for got, was, want in ((tk, bk, model.k), (tv, bv, model.v), (te, be, model.e)):
                assert np.array_equal(got[u, :nt], want[u][nf * B:]), (i, u)
                assert np.array_equal(got[u, nt:], was[u, nt:], equal_nan=True), (i, u)  # rows behind: as they were
    assert status.item() == 0
    images = units.cpu().numpy()
    used = np.zeros(len(images), bool)
    for u in range(U):
        nf = len(model.e[u]) // B
        if nf:
            used[tab[u, :nf]] = True
            cut = lambda x: x[:nf * B].reshape(nf, B, -1)  # noqa: E731
            want = Q.encode(cut(model.k[u]), cut(model.v[u]), cut(model.e[u])[..., 0])
            assert np.array_equal(images[tab[u, :nf]], want), u
    assert (images[~used] == 0xA5).all()


def test_append_turns_as_rotate_does():
    """The keys that the append turns are those of nosa_rotate, in the tail and in the blocks."""
    rng = np.random.default_rng(8)
    cfg = config(2, 4, 2, 128, "bf16")
    turn = Turn(128, 4000, some_axes("sections", 64))
    k, v = query(rng, 2, 333, 2, 128, "bf16"), query(rng, 2, 333, 2, 128, "bf16")
    pos = dev(turn.positions(rng, 2, 333))
    turned = torch.empty_like(k)
    nosa.nosa_rotate(cfg, turn.rope, pos, None, k, k_out=turned)
    got = []
    for kk, kw in ((k, dict(rope=turn.rope, positions=pos)), (turned, {})):
        units = torch.zeros(4 * 6, Q.unit_bytes(128), dtype=torch.uint8, device="cuda")
        tail = torch.zeros(4 * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
        lens = torch.zeros(4, dtype=torch.int32, device="cuda")
        nosa.nosa_quant4_append(cfg, kk, v, None, units, dev(np.arange(24).reshape(4, 6).astype(np.int32)), tail, lens, **kw)
        got.append((units, tail, lens))
    assert all(torch.equal(x, y) for x, y in zip(*got)) and got[0][0].any()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 128), ("bf16", 64)])
@pytest.mark.parametrize("n", [64, 128])
def test_append_special_values(dtype, d, n):
    """Blocks of zeros, all masked, of tiny and of huge numbers, with NaN and infinities in masked
    and in live tokens, lowest logits, one live token, equal numbers, one outlier: n = 64 and 128 take both launches."""
    names = ["zeros", "masked", "tiny", "huge", "nan masked", "nan live", "inf live", "lowest", "one token", "equal", "outlier", "powers",
             "negative zeros", "v nan live"]
    rng = np.random.default_rng(5)
    U = len(names)
    low = np.finfo(np.float32).min
    x = rng.normal(size=(U, n, 1, d))
    e = rng.normal(size=(U, n, 1)).astype(np.float32)
    v = rng.normal(size=(U, n, 1, d))
    x[0] = 0
    e[1] = -np.inf
    x[2] *= 2.0 ** -110
    x[3] *= 2.0 ** 120
    e[4, 5:9] = -np.inf
    x[4, 5], x[4, 6], x[4, 7] = np.nan, np.inf, -np.inf
    v[4, 6], v[4, 8, 0, 3] = np.nan, -np.inf
    x[5, 7, 0, 3] = np.nan
    x[6, 63, 0, d - 1] = -np.inf
    e[7] = low
    e[8] = -np.inf
    e[8, 17] = 2.0
    x[9], v[9] = 5.0, -3.0
    x[10, 11, 0, 2], v[10, 12, 0, 5] = 2.0 ** 20, -2.0 ** 25
    x[11] = 2.0 ** rng.integers(-20, 20, size=x[11].shape)
    v[11] = -(2.0 ** rng.integers(-40, 0, size=x[11].shape))
    x[12], v[12] = -0.0, -0.0
    v[13, 9, 0, 1] = np.nan
    cfg = config(U, 1, 1, d, dtype)
    nb = n // B
    units = torch.full((U * nb, Q.unit_bytes(d)), 3, dtype=torch.uint8, device="cuda")
    tab = dev(np.arange(U * nb).reshape(U, nb).astype(np.int32))
    tail = torch.zeros(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(U, dtype=torch.int32, device="cuda")
    kt, vt = dev(x, DT[dtype]), dev(v, DT[dtype])
    nosa.nosa_quant4_append(cfg, kt, vt, dev(e), units, tab, tail, lens)
    img = units.cpu().numpy().reshape(U, nb, -1)
    kf, vf = f64(kt)[:, :, 0].reshape(U, nb, B, d), f64(vt)[:, :, 0].reshape(U, nb, B, d)
    ef = e[:, :, 0].reshape(U, nb, B)
    for u, name in enumerate(names):
        want = Q.encode(kf[u], vf[u], ef[u].astype(np.float64))
        at = 71 * d + 4 * B
        sc, sw = (y[:, at:at + 8].copy().view(np.float32) for y in (img[u], want))
        assert np.array_equal(sc, sw, equal_nan=True), name
        same = [np.array_equal(np.delete(img[u, j], np.s_[at:at + 8]), np.delete(want[j], np.s_[at:at + 8])) for j in range(nb)]
        assert all(same), (name, same)


@pytest.mark.parametrize("n", [2, 200])
def test_append_leaves_what_does_not_fit(n):
    cfg = config(4, 2, 1, 64, "bf16")
    U, cap = 4, 3
    lens0 = np.array([cap * B - 1, cap * B + 1, -3, 60], np.int32)  # full, not a length, not a length, fits if n = 2
    units = torch.full((U * cap, Q.unit_bytes(64)), 7, dtype=torch.uint8, device="cuda")
    tab = np.arange(U * cap).reshape(U, cap).astype(np.int32)
    tail = torch.full((U * nosa.nosa_payload_bytes(cfg),), 9, dtype=torch.uint8, device="cuda")
    lens, status = dev(lens0), torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.randn(4, n, 1, 64, device="cuda").bfloat16()
    turn = Turn(64, 10)
    pos = np.full((1, 4, n), -9, np.int32)
    pos[:, 3] = 1  # only the last request's are read
    nosa.nosa_quant4_append(cfg, k, k, None, units, dev(tab), tail, lens, rope=turn.rope, positions=dev(pos if n == 2 else abs(pos) % 10),
                            status=status)
    fits = n == 2
    assert lens.tolist() == [lens0[0], lens0[1], lens0[2], 60 + (n if fits else 0)]
    assert status.item() == nosa.NOSA_QUANT_INDEX | nosa.NOSA_QUANT_CAPACITY
    assert (units == 7).all()
    t = tail.view(U, -1)
    assert (t[:3] == 9).all() and bool((t[3] == 9).all()) == (not fits)


def test_append_bad_entries_and_counts():
    """Destinations outside the pool are skipped and flagged, counts clamped and flagged, positions too."""
    cfg = config(3, 1, 1, 64, "f32")
    units = torch.full((2, Q.unit_bytes(64)), 3, dtype=torch.uint8, device="cuda")
    tab = dev(np.array([[2, 1], [-1, 0], [0, 0]], np.int32))
    tail = torch.zeros(3 * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    lens, status = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.randn(3, 70, 1, 64, device="cuda")
    out = torch.empty_like(lens)
    nosa.nosa_quant4_append(cfg, k, k, None, units, tab, tail, lens, lens_out=out, status=status,
                            n_new=dev(np.array([70, 99, -5], np.int32)))
    assert out.tolist() == [70, 70, 0] and lens.tolist() == [0, 0, 0]
    assert (units == 3).all() and status.item() == nosa.NOSA_QUANT_INDEX
    turn = Turn(64, 10)
    pos = np.zeros((1, 3, 70), np.int32)
    pos[0, 2, 69] = 10
    status.zero_()
    good = dev(np.array([[0], [1], [1]], np.int32))
    nosa.nosa_quant4_append(cfg, k, k, None, units, good, tail, torch.zeros_like(lens), lens_out=out, status=status, rope=turn.rope,
                            positions=dev(pos), n_new=dev(np.array([10, 64, 5], np.int32)))
    assert status.item() == 0 and out.tolist() == [10, 64, 5]
    pos[0, 1, 63] = 10
    nosa.nosa_quant4_append(cfg, k, k, None, units, good, tail, torch.zeros_like(lens), lens_out=out, status=status, rope=turn.rope,
                            positions=dev(pos), n_new=dev(np.array([10, 64, 5], np.int32)))
    assert status.item() == nosa.NOSA_QUANT_INDEX


def test_append_nothing():
    cfg = config(2, 2, 2, 64, "bf16")
    lens = dev(np.array([3, 64, 0, 70], np.int32))
    out = torch.zeros_like(lens)
    units = torch.zeros(4, Q.unit_bytes(64), dtype=torch.uint8, device="cuda")
    tail = torch.zeros(4 * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    k = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    nosa.nosa_quant4_append(cfg, k, k, None, units, dev(np.zeros((4, 2), np.int32)), tail, lens, lens_out=out)
    assert out.tolist() == [3, 64, 0, 70]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64)])
def test_read_matches_oracle(dtype, d):
    rng = np.random.default_rng(d)
    n = 9
    e = rng.normal(size=(n, B))
    e[rng.random(size=e.shape) < 0.1] = -np.inf
    e[4] = -np.inf
    img = Q.encode(rng.normal(size=(n, B, d)) + 9 * rng.normal(size=(n, 1, d)), rng.normal(size=(n, B, d)), e)
    at = 71 * d + 4 * B
    img[7, at + 4:at + 8].view(np.float32)[:] = np.nan  # values of a block that had a NaN
    cfg = config(1, 2, 1, d, dtype)
    units = dev(img)
    K, V, _, Ks, Vs = Q.decode(img, d)
    live = ~np.isneginf(e)[..., None]
    bits = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    ids = np.array([3, 8, 3, -1, 0, 4, 9, 7], np.int32)
    ok = (ids >= 0) & (ids < n)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    k, v = (torch.full((len(ids), B, d), 7.0, dtype=DT[dtype], device="cuda") for _ in range(2))
    eo = torch.full((len(ids), B), 7.0, device="cuda")
    nosa.nosa_quant4_read(cfg, units, k, v, eo, ids=dev(ids), status=status)
    assert status.item() == nosa.NOSA_QUANT_INDEX
    for got, x, size in ((k, K, Ks), (v, V, Vs)):
        want = np.where(live, x, 0.0)[ids[ok]]
        tol = np.where(live, size, 0.0)[ids[ok]] * 2.0 ** -23 + np.abs(want) * bits
        g = f64(got)
        assert np.array_equal(np.isnan(g[ok]), np.isnan(want))
        assert not np.any(np.abs(g[ok] - want) > tol)
        assert (g[~ok] == 7.0).all()
    assert np.array_equal(f64(eo)[ok], e.astype(np.float32).astype(np.float64)[ids[ok]]) and (f64(eo)[~ok] == 7.0).all()
    # parts alone, without ids, of nothing
    k2, e2 = torch.empty(5, B, d, dtype=DT[dtype], device="cuda"), torch.empty(n, B, device="cuda")
    nosa.nosa_quant4_read(cfg, units, k2)
    nosa.nosa_quant4_read(cfg, units, e_out=e2)
    nosa.nosa_quant4_read(cfg, units, v_out=v[:0], ids=dev(ids[:0]))
    assert torch.equal(k2[0], k[4]) and torch.equal(k2[3], k[0])
    assert np.array_equal(f64(e2), e.astype(np.float32).astype(np.float64))


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Cache:
    """A 4-bit cache with random contents: device arrays and their values."""

    def __init__(self, rng, dtype, batch, hq, hkv, d, lens, cap=None, masked=0.02, spare=3, scale=1.0):
        self.dims = (dtype, batch, hq, hkv, d)
        self.cfg = config(batch, hq, hkv, d, dtype)
        U = batch * hkv
        self.lens = np.asarray(lens, np.int32)
        self.cap = cap or max(1, -(-int(self.lens.max()) // B))
        nf = self.lens // B
        pool = int(nf.sum()) + spare
        perm = rng.permutation(pool)
        self.tab = np.full((U, self.cap), -1, np.int32)
        at = 0
        for u in range(U):
            self.tab[u, :nf[u]] = perm[at:at + nf[u]]
            at += nf[u]
        mean = rng.normal(size=(1, 1, d)) * np.where(np.arange(d) % 16 == 5, 4.0, 0.5)
        k = (rng.normal(size=(pool, 1, d)) * 0.5 + mean + rng.normal(size=(pool, B, d))) * scale
        v = rng.normal(size=(pool, B, d))
        e = rng.normal(size=(pool, B))
        e[rng.random(size=e.shape) < masked] = -np.inf
        self.images = Q.encode(k, v, e)
        self.tk = f64(torch.as_tensor((rng.normal(size=(U, B, d)) + mean) * scale).to(DT[dtype]))
        self.tv = f64(torch.as_tensor(rng.normal(size=(U, B, d))).to(DT[dtype]))
        self.te = rng.normal(size=(U, B)).astype(np.float32)
        self.te[rng.random(size=self.te.shape) < masked] = -np.inf

    def logits(self, u, j):
        """The logits of block j of unit u, as a view."""
        at = 71 * self.dims[4]
        return self.images[self.tab[u, j], at:at + 4 * B].view(np.float32)

    def scales(self, u, j):
        at = 71 * self.dims[4] + 4 * B
        return self.images[self.tab[u, j], at:at + 8].view(np.float32)

    def upload(self):
        dtype, _, _, _, d = self.dims
        self.units, self.t_tab, self.t_lens = dev(self.images), dev(self.tab), dev(self.lens)
        self.tail = make_tail(self.cfg, self.tk, self.tv, self.te, d, dtype)
        return self

    def tokens(self, u):
        """K, V, e of unit u's tokens in fp64 (skipped entries: masked), and the sizes that bound errors."""
        nf, nt = divmod(int(self.lens[u]), B)
        d = self.dims[4]
        ids = self.tab[u, :nf]
        ok = (ids >= 0) & (ids < len(self.images))
        K, V, e, Ks, Vs = Q.decode(self.images[np.where(ok, ids, 0)], d)
        e = np.where(ok[:, None], e, -np.inf)
        both = lambda x, t: np.concatenate([x.reshape(-1, d), t[u, :nt]])  # noqa: E731
        return (both(K, self.tk), both(V, self.tv), np.concatenate([e.ravel(), self.te[u, :nt].astype(np.float64)]),
                both(Ks, np.abs(self.tk)), both(Vs, np.abs(self.tv)))

    def run(self, q, q_len=None, mass=None, decay=1.0, **kw):
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:3], 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = nosa.nosa_quant4_attention(
            self.cfg, self.units, self.t_tab, self.tail, self.t_lens, q, out, lse=lse, mass=mass, decay=decay,
            q_len=None if q_len is None else dev(np.asarray(q_len, np.int32)), status=status, **kw)
        return out, lse, status.item()

    def check(self, q, out, lse, q_len=None, mass0=None, mass=None, decay=1.0):
        """q: the queries as the products take them (fp64, turned), or the tensor."""
        dtype, batch, hq, hkv, d = self.dims
        qf, of, lf = q if isinstance(q, np.ndarray) else f64(q), f64(out), f64(lse)
        T, G = qf.shape[1], hq // hkv
        p_bits, o_bits = (2.0 ** -11, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -21, 2.0 ** -24)
        for u in range(batch * hkv):
            b, h = divmod(u, hkv)
            n, tq = int(self.lens[u]), T if q_len is None else q_len[b]
            K, V, e, Ks, Vs = self.tokens(u)
            rows = qf[b, :tq, h * G:(h + 1) * G].reshape(tq * G, d)
            sees = np.repeat(n - tq + 1 + np.arange(tq), G)
            want, wl, w, A, S = Q.attend(rows, K, V, e, sees, Ks, Vs)
            got = of[b, :tq, h * G:(h + 1) * G].reshape(tq * G, d)
            gl = lf[b, :tq, h * G:(h + 1) * G].reshape(-1)
            empty = np.isneginf(wl)
            assert np.array_equal(np.isneginf(gl), empty), u
            assert not got[empty].any()
            dl = 2.0 ** -18 * S + 2.0 ** -22 * np.abs(np.where(empty, 0.0, wl))
            rel = 2 * dl + 2.0 ** -20 + (n / 16 + 16) * 2.0 ** -23
            tol = o_bits * np.abs(want) + (2 * p_bits + 2 * rel[:, None]) * A + 1e-30
            assert np.all(np.abs(got - want) <= tol), (u, np.max(np.abs(got - want) / tol))
            far = np.abs(gl[~empty] - wl[~empty])
            assert np.all(far <= (dl + rel)[~empty] + 2.0 ** -23 * np.abs(wl[~empty])), u
            if mass is not None:
                full = np.zeros(self.cap * B)
                full[:n] = w.sum(0)
                per = full.reshape(self.cap, B).sum(1)
                keep = np.asarray(mass0[u], np.float64) * decay if decay else 0.0
                expect = keep + per
                tol = (rel.max() if rel.size else 0.0) * per + 2.0 ** -22 * np.abs(expect) + 1e-30
                assert np.all(np.abs(mass[u] - expect) <= tol), u
            if tq < T:  # rows past the request's queries are left
                assert (of[b, tq:, h * G:(h + 1) * G] == 7.0).all() and (lf[b, tq:, h * G:(h + 1) * G] == 7.0).all()


CASES = [  # dtype, batch, hq, hkv, d, lens by request (heads differ by -h), queries
    ("bf16", 2, 8, 2, 128, [700, 64], 1), ("f32", 1, 4, 1, 64, [2031], 1), ("bf16", 3, 3, 3, 64, [1, 63, 65], 1),
    ("f32", 2, 12, 4, 128, [130, 127], 1), ("bf16", 1, 12, 2, 128, [1300], 1), ("bf16", 1, 8, 1, 64, [4000], 1),
    ("f32", 1, 2, 2, 128, [0], 1), ("bf16", 2, 8, 2, 128, [700, 3], 8), ("f32", 1, 6, 2, 64, [333], 5),
    ("bf16", 1, 8, 1, 128, [640], 32), ("f32", 1, 8, 1, 128, [200], 17), ("bf16", 1, 4, 4, 64, [129], 128),
    ("bf16", 40, 4, 4, 64, [70 + 5 * i for i in range(40)], 1), ("bf16", 2, 6, 1, 128, [190, 64], 3), ("f32", 1, 8, 2, 128, [500], 4),
    ("bf16", 300, 4, 4, 64, [37 * i % 200 for i in range(300)], 1), ("f32", 150, 8, 8, 64, [29 * i % 150 for i in range(150)], 2)]


@pytest.mark.parametrize("dtype,batch,hq,hkv,d,lens,T", CASES)
@pytest.mark.parametrize("with_mass", [False, True])
def test_attention_matches_oracle(dtype, batch, hq, hkv, d, lens, T, with_mass):
    rng = np.random.default_rng(hq * d + T)
    per_unit = [max(0, n - h) for n in lens for h in range(hkv)]
    c = Cache(rng, dtype, batch, hq, hkv, d, per_unit, cap=max(per_unit) // B + 2).upload()
    q = query(rng, batch, T, hq, d, dtype)
    m0 = rng.random(size=c.tab.shape).astype(np.float32) if with_mass else None
    mass = dev(m0) if with_mass else None
    out, lse, status = c.run(q, mass=mass, decay=0.75)
    assert status == 0
    c.check(q, out, lse, mass0=m0, mass=None if mass is None else f64(mass), decay=0.75)
    # the same workspace again, holding whatever the first call left: the same bits
    ws, m1 = c.workspace, dev(m0) if with_mass else None
    out2, lse2, _ = c.run(q, mass=m1, decay=0.75, workspace=ws)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and (mass is None or torch.equal(mass, m1))
    # and other queries right behind each other: nothing of the call before is left over
    qs = [query(rng, batch, T, hq, d, dtype) for _ in range(3)]
    res = [c.run(x, workspace=ws) if mass is None else c.run(x, mass=dev(m0), workspace=ws) for x in qs]
    c.check(qs[-1], *res[-1][:2])
    assert not torch.equal(res[0][0], res[2][0]) or not any(lens)


@pytest.mark.parametrize("dtype,hq,hkv,d,T,rot,kind,interleaved", [
    ("bf16", 8, 2, 128, 1, 128, "one", False), ("bf16", 6, 2, 64, 3, 64, "sections", False), ("f32", 4, 2, 64, 1, 32, "uneven", True),
    ("bf16", 8, 2, 128, 8, 96, "mixed", False), ("f32", 4, 1, 128, 8, 128, "one", False), ("bf16", 4, 4, 64, 1, 48, "four", False),
    ("f32", 3, 3, 128, 1, 112, "mixed", False), ("bf16", 8, 1, 128, 40, 16, "one", True), ("f32", 8, 1, 64, 9, 16, "one", False)])
def test_attention_turns_as_rotate_does(dtype, hq, hkv, d, T, rot, kind, interleaved):
    """Queries turned on the way: the same bits as queries turned before, in the blocks' products and the tail's."""
    rng = np.random.default_rng(rot + T)
    batch = 3
    c = Cache(rng, dtype, batch, hq, hkv, d, [n for n in (400, 64, 50) for _ in range(hkv)]).upload()
    turn = Turn(rot, 3000, some_axes(kind, rot // 2), interleaved)
    pos = turn.positions(rng, batch, T)
    q_len = [T, max(1, T - 1), T]
    for b in range(batch):
        pos[:, b, q_len[b]:] = 3000  # (not read)
    wide = query(rng, batch, T, hq + 2, d, dtype)
    q = wide[:, :, 1:hq + 1]  # strided rows
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass, mass2 = dev(m0), dev(m0)
    out, lse, status = c.run(q, q_len=q_len, mass=mass, rope=turn.rope, positions=dev(pos))
    assert status == 0
    c.check(turn.oracle(f64(q), pos, dtype), out, lse, q_len=q_len, mass0=m0, mass=f64(mass))
    turned = torch.empty(q.shape, dtype=q.dtype, device="cuda")
    nosa.nosa_rotate(c.cfg, turn.rope, dev(np.minimum(pos, 2999)), q, q_out=turned)
    out2, lse2, _ = c.run(turned, q_len=q_len, mass=mass2)
    assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(mass, mass2)
    pos[0, 0, 0] = -1
    pos[:, 0, 1:] = 5
    assert c.run(q, q_len=q_len, rope=turn.rope, positions=dev(pos))[2] == nosa.NOSA_QUANT_INDEX


@pytest.mark.parametrize("dtype,hq,hkv,d,T", [
    ("bf16", 6, 3, 128, 1), ("bf16", 6, 3, 64, 1), ("f32", 6, 3, 128, 1), ("f32", 6, 3, 64, 1), ("bf16", 8, 2, 128, 4),
    ("bf16", 8, 2, 64, 4), ("bf16", 8, 2, 128, 8), ("f32", 8, 2, 64, 8), ("f32", 8, 2, 128, 7), ("f32", 4, 1, 128, 3)])
def test_attention_long_rings(dtype, hq, hkv, d, T):
    """Enough blocks that every CTA goes round its ring several times and crosses units; the
    tables name the units of a small pool many times."""
    rng = np.random.default_rng(T * d)
    batch = 4
    c = Cache(rng, dtype, batch, hq, hkv, d, [64 * 70 + 5] * (batch * hkv))
    lens = np.array([64 * 1500 + 40, 64 * 900, 70, 64 * 2100 + 1, 64 * 30, 64 * 1200 + 63, 1, 64 * 800, 64 * 999 + 2,
                     64 * 640, 64 * 333 + 33, 64 * 1024][:batch * hkv], np.int32)
    c.cap = 2101
    c.lens = lens
    c.tab = rng.integers(0, len(c.images), size=(len(lens), c.cap)).astype(np.int32)
    c.upload()
    q = query(rng, batch, T, hq, d, dtype)
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass, decay=0.5)
    assert status == 0
    c.check(q, out, lse, mass0=m0, mass=f64(mass), decay=0.5)
    for _ in range(20):  # and again, many times, with the same result
        m1 = dev(m0)
        out2, lse2, status = c.run(q, mass=m1, decay=0.5, workspace=c.workspace)
        assert status == 0 and torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(mass, m1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_query_counts_and_strides(dtype):
    rng = np.random.default_rng(9)
    batch, hq, hkv, d, T = 4, 8, 2, 128, 6
    lens = [500, 129, 3, 64]
    c = Cache(rng, dtype, batch, hq, hkv, d, [n for n in lens for _ in range(hkv)]).upload()
    q_len = [6, 1, 5, 0]  # request 2: more queries than tokens, the first rows see nothing
    wide = query(rng, batch, T, hq + 2 * hkv, d, dtype)
    q = wide[:, :, hkv:hkv + hq]
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, q_len=q_len, mass=mass, decay=1.0)
    assert status == 0
    c.check(q, out, lse, q_len=q_len, mass0=m0, mass=f64(mass))
    assert not f64(out)[2, :2].any()
    same = q[:, :1, :1].expand(batch, T, hq, d)  # strides of zero
    out, lse, _ = c.run(same)
    c.check(same, out, lse)
    _, _, status = c.run(q, q_len=[6, 7, -1, 6])  # counts out of range are clamped and flagged
    assert status == nosa.NOSA_QUANT_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 2, 9])
def test_attention_masks(dtype, d, T):
    """Units with every token masked, with only the tail or only one block visible, with lowest
    logits everywhere, with NaN and infinities in masked places of the tail and of blocks (steps, zeros,
    codes of masked tokens), with a masked block whose scales are NaN."""
    rng = np.random.default_rng(21)
    hq = 8
    names = ["all masked", "tail only", "one block", "lowest", "nan masked", "block masked", "lowest but one", "masked steps"]
    U = len(names)
    c = Cache(rng, dtype, U, hq, 1, d, [300] * U, masked=0.0)
    low = np.finfo(np.float32).min
    for j in range(4):
        for u in (0, 1, 2):
            if not (u == 2 and j == 2):
                c.logits(u, j)[:] = -np.inf
        for u in (3, 6):
            c.logits(u, j)[:] = low
    c.logits(6, 1)[:] = np.where(np.arange(B) == 5, 0.5, low)
    c.te[0] = c.te[2] = -np.inf
    c.te[3] = c.te[6] = low
    c.te[4, 3:8] = -np.inf
    c.tk[4, 3:5] = np.nan
    c.tv[4, 4:8] = np.inf
    c.scales(5, 1)[:] = np.nan
    c.logits(5, 1)[:] = -np.inf
    (kb, ks), (vb, vs) = Q.code_places(d)
    _, _, vstep, vzero = Q.places(d)
    gone = {0: [17], 1: [0, 5, 10, 15, 18, 35, 52, 63], 2: list(range(B)), 3: list(range(1, B))}
    clean = c.images.copy()
    for j, tokens in gone.items():
        c.logits(7, j)[tokens] = -np.inf
        clean[c.tab[7, j]] = c.images[c.tab[7, j]]
        row = c.images[c.tab[7, j]]
        for i, t in enumerate(tokens):
            for at, bits in ((vstep[t], [0x7E00, 0x7C00, 0xFC00][i % 3]), (vzero[t], [0xFC00, 0x7E00, 0x3C00][i % 3])):
                row[at], row[at + 1] = bits & 255, bits >> 8
            row[vb[t]] |= (15 << vs[t]).astype(np.uint8)
            row[kb[t]] |= (15 << ks[t]).astype(np.uint8)
        if j == 2:  # no token of the block counts: nor do its channels' steps and zeros
            row[64 * d:67 * d] = 0x7E
    c.upload()
    assert torch.isnan(c.tail.view(DT[dtype])).any()
    q = query(rng, U, T, hq, d, dtype)
    m0 = np.zeros(c.tab.shape, np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass)
    assert status == 0
    dirty = c.images
    c.images = clean
    for j in gone:
        dirty_e = dirty[c.tab[7, j], 71 * d:71 * d + 4 * B]
        clean[c.tab[7, j], 71 * d:71 * d + 4 * B] = dirty_e
    c.scales(5, 1)[:] = 1.0
    c.tk[4, 3:8], c.tv[4, 3:8] = 0.0, 0.0  # masked: not looked at
    c.check(q, out, lse, mass0=m0, mass=f64(mass))
    assert torch.equal(c.units, dev(dirty))  # the cache itself keeps its bytes


def test_attention_nan_reaches_only_its_rows():
    """A live NaN (scale) makes the rows that see it NaN and no others; a NaN query its own row."""
    rng = np.random.default_rng(2)
    c = Cache(rng, "bf16", 3, 4, 1, 64, [200, 200, 200])
    c.scales(1, 1)[0] = np.nan
    c.upload()
    q = query(rng, 3, 1, 4, 64, "bf16")
    q[2, 0, 1, 5] = float("nan")
    out, lse, status = c.run(q)
    assert status == 0
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert not torch.isnan(out[0]).any() and not torch.isnan(lse[0]).any()
    assert torch.isnan(out[2, 0, 1]).all() and not torch.isnan(out[2, 0, [0, 2, 3]]).any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,T", [(4, 2), (1, 70)])
def test_attention_value_nan_reaches_the_rows_that_see_it(dtype, hq, T):
    """A value's step that is no number, in a token that is not masked, reaches the rows that see that
    token, in its run of dims, and no others; a NaN value of the tail its rows."""
    rng = np.random.default_rng(33)
    d, n = 128, 192
    c = Cache(rng, dtype, 1, hq, 1, d, [n], masked=0.0)
    at = Q.places(d)[2][B - 1, 1]  # the newest token, the second run
    row = c.images[c.tab[0, 2]]
    row[at], row[at + 1] = 0, 0x7E
    c.upload()
    q = query(rng, 1, T, hq, d, dtype)
    out, lse, status = c.run(q)
    assert status == 0
    nan = torch.isnan(out[0])
    assert nan[-1, :, 64:].all() and not nan[-1, :, :64].any() and not nan[:-1].any() and not torch.isnan(lse).any()


def test_attention_large_and_small_queries():
    """Queries near the ends of the bf16 range, keys of tiny and huge blocks: logits stay what they are."""
    rng = np.random.default_rng(6)
    c = Cache(rng, "bf16", 1, 4, 1, 64, [150], scale=2.0 ** -60).upload()
    q = query(rng, 1, 1, 4, 64, "bf16")
    q[:, :, 0] *= 2.0 ** 60
    q[:, :, 1] *= 2.0 ** -100
    q[:, :, 2] *= 2.0 ** 59
    out, lse, status = c.run(q)
    assert status == 0
    c.check(q, out, lse)


@pytest.mark.parametrize("d,n", [(64, 704), (128, 704), (64, 16384), (128, 16384)])
def test_attention_fp32_outputs_in_the_norm(d, n):
    """fp32 outputs keep fp32's bits in the norm too, where values of both signs nearly cancel.

    Each weight is off by a few independent roundings (its two 11-bit terms and their products with a step,
    2^-22 each; the exponential, 2^-22; its logit, some 2^-22), so sum w_j v_j of independent v_j is off by 2^-21
    of its norm or so, and with the sums' own additions by 2^-19 at most. Sums that cut off at the size of
    sum w_j |v_j| would show: that is sqrt(n) times the output here."""
    rng = np.random.default_rng(d + n)
    c = Cache(rng, "f32", 2, 4, 1, d, [n] * 2, cap=n // B + 1, masked=0.0).upload()
    q = query(rng, 2, 1, 4, d, "f32")
    out, lse, status = c.run(q)
    assert status == 0
    for u in range(2):
        K, V, e, Ks, Vs = c.tokens(u)
        want, wl = Q.attend(f64(q)[u, 0], K, V, e, np.full(4, n), Ks, Vs)[:2]
        got = f64(out)[u, 0]
        assert np.linalg.norm(got - want) <= 2.0 ** -19 * np.linalg.norm(want), u


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
def test_attention_logits_of_queries_with_large_elements(dtype, d):
    """An element in 16 of a query is 512 times the others, the keys are not zero there: the lesser products
    are not cut off at the size of the larger operands.

    The codes are fp16 operands whose exponents are at most 2^6 too large for a code of 15; a sum of 16 products
    is cut off 2^-24 below its largest exponent, so 2^-18 q step for each of the 15 lesser ones, and those are
    independent: 2^-17 q step for d / 16 sums of 16, of which S is at least 7 d / 16 q step (step n + |zero| of
    a normal sample's 16 levels): 2^-19.8 S / sqrt(d / 16), at most 2^-20 S for what the lse of a few large logits shows."""
    rng = np.random.default_rng(d)
    c = Cache(rng, dtype, 4, 8, 1, d, [704] * 4, masked=0.0).upload()
    q = query(rng, 4, 1, 8, d, dtype)
    q[..., 3::16] *= 512
    out, lse, status = c.run(q)
    assert status == 0
    for u in range(4):
        K, V, e, Ks, Vs = c.tokens(u)
        want, wl, w, A, S = Q.attend(f64(q)[u, 0], K, V, e, np.full(8, 704), Ks, Vs)
        assert np.all(np.abs(f64(lse)[u, 0] - wl) <= 2.0 ** -20 * S + 2.0 ** -23 * np.abs(wl)), u
    c.check(q, out, lse)


@pytest.mark.parametrize("dtype,d,T", [("bf16", 64, 1), ("bf16", 128, 1), ("f32", 64, 1), ("f32", 128, 1), ("bf16", 128, 8), ("f32", 128, 4)])
def test_attention_queries_with_an_outlier(dtype, d, T):
    """One element of 30 000 in a query meets keys of zero: the logits keep the others' bits."""
    rng = np.random.default_rng(41)
    c = Cache(rng, dtype, 1, 4, 1, d, [700], masked=0.0)
    k = rng.normal(size=(len(c.images), B, d))
    k[..., 3] = 0.0
    c.images = Q.encode(k, rng.normal(size=k.shape), rng.normal(size=k.shape[:2]))
    c.tk[..., 3] = 0.0
    c.upload()
    q = query(rng, 1, T, 4, d, dtype)
    q[..., 3] = 30000.0
    out, lse, status = c.run(q)
    assert status == 0
    c.check(q, out, lse)


def test_attention_bad_entries_and_lengths():
    rng = np.random.default_rng(8)
    c = Cache(rng, "bf16", 2, 4, 1, 64, [300, 200])
    c.tab[0, 1], c.tab[1, 0] = len(c.images), -7
    c.upload()
    q = query(rng, 2, 1, 4, 64, "bf16")
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass)
    assert status == nosa.NOSA_QUANT_INDEX
    c.check(q, out, lse, mass0=m0, mass=f64(mass))  # skipped blocks weigh nothing
    c.t_lens = dev(np.array([300, c.cap * B + 1], np.int32))
    out, lse, status = c.run(q)
    assert status == nosa.NOSA_QUANT_INDEX and not out[1].any() and torch.isneginf(lse[1]).all()


def test_attention_mass_overwrites_with_decay_zero():
    rng = np.random.default_rng(10)
    c = Cache(rng, "f32", 1, 4, 2, 64, [130, 64]).upload()
    q = query(rng, 1, 1, 4, 64, "f32")
    mass = torch.full(c.tab.shape, float("nan"), device="cuda")
    out, lse, _ = c.run(q, mass=mass, decay=0.0)
    m0 = np.zeros(c.tab.shape, np.float32)
    assert not f64(mass)[1, 1:].any()  # past the last block: nothing
    c.check(q, out, lse, mass0=m0, mass=f64(mass), decay=0.0)


def test_units_past_four_gib():
    """Table entries and ids whose byte offset passes 2^32."""
    rng = np.random.default_rng(12)
    d = 128
    n = 2 ** 32 // Q.unit_bytes(d) + 40
    c = Cache(rng, "bf16", 1, 4, 1, d, [200])
    pool = torch.empty(n, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
    at = np.array([n - 1, 5, n - 30])
    pool[dev(at)] = dev(c.images[c.tab[0, :3]])
    c.upload()
    c.units, c.t_tab = pool, dev(np.concatenate([at, [-1]])[None].astype(np.int32))
    q = query(rng, 1, 1, 4, d, "bf16")
    out, lse, status = c.run(q)
    assert status == 0
    c.check(q, out, lse)
    # the append there, and reading it back
    cfg = c.cfg
    lens = dev(np.array([0], np.int32))
    tail = torch.zeros(nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    k = torch.randn(1, 64, 1, d, device="cuda").bfloat16()
    nosa.nosa_quant4_append(cfg, k, k, None, pool, dev(np.array([[n - 2]], np.int32)), tail, lens)
    want = Q.encode(f64(k)[:, :, 0], f64(k)[:, :, 0], np.zeros((1, 64)))
    assert np.array_equal(pool[n - 2:n - 1].cpu().numpy(), want)
    back = torch.empty(1, B, d, dtype=torch.bfloat16, device="cuda")
    nosa.nosa_quant4_read(cfg, pool, v_out=back, ids=dev(np.array([n - 2], np.int32)))
    assert np.all(np.abs(f64(back) - Q.decode(want, d)[1]) <= np.abs(Q.decode(want, d)[1]) * 2.0 ** -8 + Q.decode(want, d)[4] * 2.0 ** -23)


def test_attention_on_two_streams():
    """Two calls at once, each with its own workspace, on streams that are not the current one."""
    rng = np.random.default_rng(14)
    caches = [Cache(rng, "bf16", 4, 8, 2, 128, [900 - 100 * i] * 8).upload() for i in range(2)]
    qs = [query(rng, 4, 1, 8, 128, "bf16") for _ in caches]
    streams = [torch.cuda.Stream() for _ in caches]
    torch.cuda.synchronize()
    res = []
    for _ in range(5):
        res = [c.run(q, stream=s)[:2] + (s,) for c, q, s in zip(caches, qs, streams)]
    torch.cuda.synchronize()
    for c, q, (out, lse, _) in zip(caches, qs, res):
        c.check(q, out, lse)


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured: rotation, append, attention, reading back, eviction."""
    code = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import test_quant4_gpu as t
nosa = t.nosa
rng = np.random.default_rng(3)
c = t.Cache(rng, "f32", 1, 4, 2, 64, [300, 100], cap=6).upload()
q = t.query(rng, 1, 4, 4, 64, "f32")
turn = t.Turn(64, 500)
pos = turn.positions(rng, 1, 4)
tpos, kpos = t.dev(pos), t.dev(turn.positions(rng, 1, 70))
out, lse, out2 = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda"), torch.empty_like(q)
mass = torch.zeros(c.tab.shape, device="cuda")
k = t.query(rng, 1, 70, 2, 64, "f32")
ws = torch.empty(nosa.nosa_quant4_attention_workspace_bytes(c.cfg, c.cap, 4, True), dtype=torch.uint8, device="cuda")
units = torch.zeros(len(c.images) + 6, c.images.shape[1], dtype=torch.uint8, device="cuda")
units[:len(c.images)] = c.units
c.t_tab[0, 4:] = torch.arange(2, dtype=torch.int32, device="cuda") + len(c.images)
c.t_tab[1, 1:] = torch.arange(5, dtype=torch.int32, device="cuda") + len(c.images) + 1
c.t_tab[0, 5] = len(c.images)
back = torch.empty(1, 64, 64, device="cuda")
ids = torch.tensor([len(c.images)], dtype=torch.int32, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
lens = c.t_lens.clone()
with torch.cuda.graph(g):
    nosa.nosa_quant4_attention(c.cfg, units, c.t_tab, c.tail, lens, q, out, lse=lse, mass=mass, workspace=ws, rope=turn.rope, positions=tpos)
    nosa.nosa_rotate(c.cfg, turn.rope, tpos, q, q_out=out2)
    nosa.nosa_quant4_append(c.cfg, k, k, None, units, c.t_tab, c.tail, lens, rope=turn.rope, positions=kpos)
    nosa.nosa_quant4_read(c.cfg, units, back, ids=ids)
    nosa.nosa_quant_evict(c.cfg, 2, 1, c.t_tab, mass, lens)
g.replay()
torch.cuda.synchronize()
want = turn.oracle(t.f64(q), pos, "f32")
assert np.array_equal(t.f64(out2), want)
c.check(want, out, lse)
assert back.any()
assert lens.tolist() == [64 * 2 + (300 + 70) %% 64, 64 * 2 + (100 + 70) %% 64], lens.tolist()
print("ok")
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("dtype,batch,hq,hkv,d,T,n,cap", [
    ("bf16", 2, 8, 2, 128, 1, 700, 11), ("bf16", 2, 8, 2, 64, 1, 700, 600), ("f32", 3, 4, 1, 64, 1, 400, 7), ("f32", 1, 4, 2, 128, 3, 999, 16),
    ("bf16", 2, 8, 2, 128, 12, 900, 15), ("f32", 2, 8, 2, 64, 8, 300, 5), ("bf16", 300, 4, 4, 64, 1, 130, 3), ("bf16", 2, 8, 2, 128, 3, 200, 4)])
def test_attention_wait_that_gives_up(dtype, batch, hq, hkv, d, T, n, cap, turned, monkeypatch):
    """Waits that give up at once (set on the host): the status says so, the rows that exist are
    NaN (every unit has blocks), the accumulated weights stay, the kernels end, and the next call is right."""
    rng = np.random.default_rng(61)
    c = Cache(rng, dtype, batch, hq, hkv, d, [n - h for _ in range(batch) for h in range(hkv)], cap=cap).upload()
    q = query(rng, batch, T, hq, d, dtype)
    turn = Turn(d, 1000)
    pos = turn.positions(rng, batch, T)
    kw = dict(rope=turn.rope, positions=dev(pos)) if turned else {}
    q_len = [T] * (batch - 1) + [max(1, T - 1)]
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    c.run(q, q_len=q_len, mass=dev(m0), **kw)
    ws = c.workspace
    monkeypatch.setenv("NOSA_INJECT_FAIL", "wait")
    for _ in range(3):
        out, lse, status = c.run(q, q_len=q_len, mass=mass, decay=0.5, workspace=ws, **kw)
        assert status == nosa.NOSA_QUANT_WAIT
        for b in range(batch):
            assert torch.isnan(out[b, :q_len[b]]).all() and torch.isnan(lse[b, :q_len[b]]).all()
            assert (out[b, q_len[b]:] == 7).all() and (lse[b, q_len[b]:] == 7).all()
        assert np.array_equal(mass.cpu().numpy(), m0)
    monkeypatch.delenv("NOSA_INJECT_FAIL")
    out, lse, status = c.run(q, q_len=q_len, mass=mass, decay=0.5, workspace=ws, **kw)
    assert status == 0
    c.check(turn.oracle(f64(q), pos, dtype) if turned else q, out, lse, q_len=q_len, mass0=m0, mass=f64(mass), decay=0.5)


@pytest.mark.parametrize("dtype,batch,hq,hkv,d,cap", [("bf16", 64, 16, 8, 64, 4), ("f32", 40, 8, 8, 128, 4), ("bf16", 160, 24, 8, 128, 200),
                                                      ("f32", 300, 4, 4, 64, 140)])
def test_calls_behind_each_other_read_what_the_last_one_wrote(dtype, batch, hq, hkv, d, cap):
    """Steps of append, attention, reading back, rotation and eviction over many units, whose lengths share
    cache lines, queries and keys turned by positions that change in place: queued without a pause and
    with the GPU waited for after every call, the bits are the same. A masked token's step is no number, so
    that its part is gone through again."""
    rng = np.random.default_rng(71)
    U = batch * hkv
    cfg = config(batch, hq, hkv, d, dtype)
    turn = Turn(d, 999)
    steps = 16
    ins = [(query(rng, batch, 1, hkv, d, dtype, 1.0), query(rng, batch, 1, hkv, d, dtype, 1.0), query(rng, batch, 1, hq, d, dtype),
            dev(turn.positions(rng, batch, 1))) for _ in range(steps)]
    prompt = query(rng, batch, 3 * B, hkv, d, dtype, 1.0)
    e = rng.normal(size=(batch, 3 * B, hkv)).astype(np.float32)
    e[:, 7] = -np.inf
    e, p_pos = dev(e), dev(turn.positions(rng, batch, 3 * B))
    n_new = dev(rng.integers(1, 3 * B - 1, size=batch).astype(np.int32))
    at = torch.as_tensor(Q.places(d)[2][7], device="cuda")

    def loop(pause):
        done = torch.cuda.synchronize if pause else lambda: None
        units = torch.zeros(U * 4, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
        tab = torch.zeros(U, cap, dtype=torch.int32, device="cuda")
        tab[:, :4] = torch.arange(U * 4, dtype=torch.int32, device="cuda").view(U, 4)
        tail = torch.zeros(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
        lens, mass = torch.zeros(U, dtype=torch.int32, device="cuda"), torch.zeros(U, cap, device="cuda")
        ws = torch.zeros(nosa.nosa_quant4_attention_workspace_bytes(cfg, cap, 1, True), dtype=torch.uint8, device="cuda")
        outs = [(torch.empty_like(ins[0][2]), torch.empty(batch, 1, hq, device="cuda"), torch.empty_like(ins[0][2]),
                 torch.empty(U * 4, B, d, dtype=DT[dtype], device="cuda")) for _ in range(steps)]
        pos = torch.zeros_like(ins[0][3])
        torch.cuda.synchronize()
        nosa.nosa_quant4_append(cfg, prompt, prompt, e, units, tab, tail, lens, n_new=n_new, rope=turn.rope, positions=p_pos)
        done()
        units.view(U, 4, -1)[:, 0, at + 1] |= 0x7E  # the masked token of the first block, if it is full: no number
        done()
        for (k, v, q, p), (out, lse, turned, back) in zip(ins, outs):
            pos.copy_(p)
            done()
            nosa.nosa_quant4_append(cfg, k, v, None, units, tab, tail, lens, rope=turn.rope, positions=pos)
            done()
            nosa.nosa_quant4_attention(cfg, units, tab, tail, lens, q, out, lse=lse, mass=mass, decay=0.9, rope=turn.rope, positions=pos,
                                       workspace=ws)
            done()
            nosa.nosa_rotate(cfg, turn.rope, pos, out, q_out=turned)
            done()
            nosa.nosa_quant4_read(cfg, units, back)
            done()
            nosa.nosa_quant_evict(cfg, 2, 1, tab, mass, lens)
            done()
        torch.cuda.synchronize()
        return [x for four in outs for x in four] + [mass, lens, tail, units]

    want = loop(True)
    assert not torch.isnan(want[0]).any()
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(want, loop(False)))


@pytest.mark.parametrize("dtype,hq,hkv,d,T,n", [("bf16", 8, 8, 64, 1, 70), ("bf16", 16, 4, 128, 1, 900), ("f32", 8, 2, 64, 4, 300), ("f32", 8, 4, 128, 1, 64)])
def test_attention_queries_written_by_the_call_before(dtype, hq, hkv, d, T, n):
    """Each call's queries are the outputs of the call before it, in two buffers that are written again
    and again, turned on the way: queued without a pause and with one, the bits are the same."""
    rng = np.random.default_rng(73)
    c = Cache(rng, dtype, 20, hq, hkv, d, [n] * (20 * hkv)).upload()
    first = query(rng, 20, T, hq, d, dtype)
    ws = torch.empty(nosa.nosa_quant4_attention_workspace_bytes(c.cfg, c.cap, T), dtype=torch.uint8, device="cuda")
    turn = Turn(d, 60)
    pos = dev(turn.positions(rng, 20, T))

    def chain(pause):
        a, b, seen = first.clone(), torch.empty_like(first), []
        for i in range(40):
            nosa.nosa_quant4_attention(c.cfg, c.units, c.t_tab, c.tail, c.t_lens, a, b, rope=turn.rope, positions=pos, workspace=ws)
            if pause:
                torch.cuda.synchronize()
            a, b = b, a
            if i % 8 == 7:
                seen.append(a.clone())
        torch.cuda.synchronize()
        return seen

    want = chain(True)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(want, chain(False)))


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128)])
def test_attention_the_longest_table(dtype, d):
    """16384 table entries of a few units named again and again, all rows of a request."""
    rng = np.random.default_rng(81)
    c = Cache(rng, dtype, 1, 4, 1, d, [64 * 40 + 7])
    c.cap = 16384
    c.lens = np.array([64 * 16383 + 50], np.int32)
    c.tab = rng.integers(0, len(c.images), size=(1, c.cap)).astype(np.int32)
    c.upload()
    q = query(rng, 1, 2, 4, d, dtype)
    m0 = np.zeros(c.tab.shape, np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass)
    assert status == 0
    c.check(q, out, lse, mass0=m0, mass=f64(mass))


def test_rotate_in_a_graph_on_a_stream_of_its_own():
    """A captured rotation, forth and back, replayed while the inputs change in place."""
    rng = np.random.default_rng(83)
    turn = Turn(128, 500, some_axes("sections", 64))
    cfg = config(2, 8, 2, 128, "bf16")
    q, k = query(rng, 2, 40, 8, 128, "bf16"), query(rng, 2, 40, 2, 128, "bf16")
    pos = dev(turn.positions(rng, 2, 40))
    qo, ko, back = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    g, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=stream):
        nosa.nosa_rotate(cfg, turn.rope, pos, q, k, q_out=qo, k_out=ko)
        nosa.nosa_rotate(cfg, turn.rope, pos, qo, q_out=back, backward=True)
    for _ in range(3):
        q.copy_(query(rng, 2, 40, 8, 128, "bf16"))
        p = turn.positions(rng, 2, 40)
        pos.copy_(dev(p))
        g.replay()
        torch.cuda.synchronize()
        want = turn.oracle(f64(q), p, "bf16")
        assert np.array_equal(f64(qo), want) and np.array_equal(f64(ko), turn.oracle(f64(k), p, "bf16"))
        assert np.array_equal(f64(back), turn.oracle(want, p, "bf16", True))


# ---------------------------------------------------------------------------
# all of them, as a generation uses them
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,batch,hq,hkv,d,kind", [("bf16", 2, 8, 2, 128, "one"), ("f32", 1, 4, 2, 64, "sections")])
def test_generation_loop_in_a_graph(dtype, batch, hq, hkv, d, kind):
    """Prompt, observation, first eviction, then captured steps (append, attention, eviction), keys and
    queries turned on the way, replayed past several block ends: outputs, weights, lengths and stored
    tokens against a model that keeps every turned token; two graphs share the workspace."""
    rng = np.random.default_rng(d)
    U = batch * hkv
    budget, recent, cap, decay = 4, 1, 9, 0.9
    cfg = config(batch, hq, hkv, d, dtype)
    turn = Turn(d, 2000, some_axes(kind, d // 2))
    units = torch.zeros(U * cap, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
    tab = dev(rng.permutation(U * cap).reshape(U, cap).astype(np.int32))
    tail = torch.zeros(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(U, dtype=torch.int32, device="cuda")
    mass = torch.zeros(U, cap, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    model, coded = Model(U, d), Model(U, d)  # the tokens, and what the cache should hold of them
    weight = [np.zeros(cap, np.float64) for _ in range(U)]
    seen = [0]

    def tokens(n):
        k, v = (query(rng, batch, n, hkv, d, dtype, 1.0) for _ in range(2))
        return k, v, dev(rng.normal(size=(batch, n, hkv)).astype(np.float32)), new_positions(n)

    def new_positions(n):
        p = np.broadcast_to(seen[0] + np.arange(n), (batch, n))
        p = np.stack([p] if turn.n_axes == 1 else [p // 30, p // 6 % 5, p % 6]).astype(np.int32)
        return dev(p)

    def model_append(k, v, e, pos):
        kt = turn.oracle(f64(k), pos.cpu().numpy(), dtype)
        for u in range(U):
            b, h = divmod(u, hkv)
            old = len(model.e[u])
            model.add(u, kt[b, :, h], f64(v)[b, :, h], f64(e)[b, :, h])
            coded.add(u, kt[b, :, h], f64(v)[b, :, h], f64(e)[b, :, h])
            for j in range(old // B, len(model.e[u]) // B):
                p = slice(j * B, j * B + B)
                K, V, _, _, _ = Q.decode(Q.encode(model.k[u][None, p], model.v[u][None, p], model.e[u][None, p]), d)
                coded.k[u][p], coded.v[u][p] = K[0], V[0]
        seen[0] += k.shape[1]

    def model_attend(q, pos, out, lse):
        c = Cache.__new__(Cache)
        c.dims, c.cfg, c.cap = (dtype, batch, hq, hkv, d), cfg, cap
        c.images, c.tab, c.lens = units.cpu().numpy(), tab.cpu().numpy(), lens.cpu().numpy()
        c.tk, c.tv, te = tail_arrays(cfg, tail, d, dtype)
        c.te = te.astype(np.float32)
        m0 = np.stack(weight).astype(np.float32)
        got = f64(mass)
        c.check(turn.oracle(f64(q), pos.cpu().numpy(), dtype), out, lse, mass0=m0, mass=got, decay=decay)
        for u in range(U):  # what is stored is what was appended
            assert int(c.lens[u]) == len(model.e[u])
            K, V, e, _, _ = c.tokens(u)
            assert np.array_equal(e, model.e[u]) and np.array_equal(K, coded.k[u]) and np.array_equal(V, coded.v[u])
            weight[u] = got[u].copy()
        assert status.item() == 0

    def model_evict():
        for u in range(U):
            n = len(model.e[u])
            _, wm, wn, order = evict_oracle(np.arange(cap), weight[u].astype(np.float32), n, budget, recent)
            nf, kept = n // B, wn // B
            take = np.concatenate([np.arange(B) + B * j for j in order[:kept]] + [np.arange(nf * B, n)]).astype(int)
            for m in (model, coded):
                m.k[u], m.v[u], m.e[u] = m.k[u][take], m.v[u][take], m.e[u][take]
            weight[u] = wm.astype(np.float64)
            assert lens[u].item() == wn

    # the prompt, its last 8 tokens' look back, the first eviction
    k, v, e, pos = tokens(8 * B + 21)
    nosa.nosa_quant4_append(cfg, k, v, e, units, tab, tail, lens, rope=turn.rope, positions=pos, status=status)
    model_append(k, v, e, pos)
    q = query(rng, batch, 8, hq, d, dtype)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    qpos = pos[:, :, -8:].contiguous()
    nosa.nosa_quant4_attention(cfg, units, tab, tail, lens, q, out, lse=lse, mass=mass, decay=decay, rope=turn.rope, positions=qpos,
                               status=status)
    model_attend(q, qpos, out, lse)
    nosa.nosa_quant_evict(cfg, budget, recent, tab, mass, lens, status=status)
    model_evict()

    # one step, captured twice on a stream of its own; the graphs alternate and share the workspace
    ws = torch.empty(nosa.nosa_quant4_attention_workspace_bytes(cfg, cap, 1, True), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    bufs, graphs = [], []
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        k, v, e, pos = tokens(1)
        q = query(rng, batch, 1, hq, d, dtype)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            nosa.nosa_quant4_append(cfg, k, v, e, units, tab, tail, lens, rope=turn.rope, positions=pos, status=status)
            nosa.nosa_quant4_attention(cfg, units, tab, tail, lens, q, out, lse=lse, mass=mass, decay=decay,
                                       rope=turn.rope, positions=pos, workspace=ws, status=status)
        bufs.append((k, v, e, pos, q, out, lse))
        graphs.append(g)
    evict = torch.cuda.CUDAGraph()
    with torch.cuda.graph(evict, stream=stream):
        nosa.nosa_quant_evict(cfg, budget, recent, tab, mass, lens, status=status)
    for step in range(3 * B):
        k, v, e, pos, q, out, lse = bufs[step % 2]
        for dst, src in zip((k, v, e, pos), tokens(1)):
            dst.copy_(src)
        q.copy_(query(rng, batch, 1, hq, d, dtype))
        graphs[step % 2].replay()
        model_append(k, v, e, pos)
        if step % 5 == 0 or len(model.e[0]) % B in (0, 1, 63):
            torch.cuda.synchronize()
            model_attend(q, pos, out, lse)
        else:
            got = f64(mass)
            for u in range(U):
                weight[u] = got[u].copy()
        evict.replay()
        model_evict()
    assert status.item() == 0


def test_binding_refusals():
    """Wrong types, shapes, strides, sizes, devices and alignments are refused before anything runs."""
    cfg = config(2, 4, 2, 64, "bf16")
    U, cap, bf = 4, 3, torch.bfloat16
    z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    units, tab = z(6, Q.unit_bytes(64), dtype=torch.uint8), z(U, cap, dtype=torch.int32)
    tail, lens = z(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8), z(U, dtype=torch.int32)
    k, q, mass = z(2, 5, 2, 64, dtype=bf), z(2, 5, 4, 64, dtype=bf), z(U, cap)
    out = torch.empty_like(q)
    ws = z(nosa.nosa_quant4_attention_workspace_bytes(cfg, cap, 5, True), dtype=torch.uint8)
    rope, pos = nosa.nosa_rope(z(9, 32, 2)), z(2, 5, dtype=torch.int32)
    two, wide = nosa.nosa_rope(z(9, 32, 2), axes=[0] * 31 + [1]), z(2, 5, 2, 72, dtype=bf)
    back = z(3, 64, 64, dtype=bf)

    def append(k=k, v=k, e=None, units=units, tab=tab, tail=tail, lens=lens, **kw):
        nosa.nosa_quant4_append(cfg, k, v, e, units, tab, tail, lens, **kw)

    def attention(units=units, tab=tab, tail=tail, lens=lens, q=q, out=out, workspace=ws, **kw):
        nosa.nosa_quant4_attention(cfg, units, tab, tail, lens, q, out, workspace=workspace, **kw)

    def rotate(rope=rope, pos=pos, q=q, k=k, **kw):
        nosa.nosa_rotate(cfg, rope, pos, q, k, **kw)

    def read(units=units, k_out=back, **kw):
        nosa.nosa_quant4_read(cfg, units, k_out, **kw)

    eight = z(6, nosa.nosa_quant_unit_bytes(cfg), dtype=torch.uint8)
    other = config(2, 4, 2, 64, "bf16")
    other.device = 1
    bad = [
        lambda: append(k=k.float()), lambda: append(v=k[:, :4]), lambda: append(k=wide[..., 1:65]), lambda: append(e=z(2, 5, 4)),
        lambda: append(units=eight), lambda: append(tail=tail[:-256]), lambda: append(lens=lens[:2]), lambda: append(tab=tab.long()),
        lambda: append(rope=rope), lambda: append(positions=pos), lambda: append(rope=rope, positions=pos[:, :4]),
        lambda: append(rope=rope, positions=pos.long()), lambda: append(rope=two, positions=pos), lambda: append(rope=5, positions=pos),
        lambda: append(rope=rope, positions=[0]), lambda: append(rope=rope, positions=pos.cpu()),
        lambda: attention(units=eight), lambda: attention(q=q.float()), lambda: attention(out=q), lambda: attention(mass=z(U, cap + 1)),
        lambda: attention(mass=mass, decay=2.0), lambda: attention(mass=mass, workspace=ws[:256]), lambda: attention(workspace=ws[16:]),
        lambda: attention(rope=rope), lambda: attention(rope=two, positions=pos), lambda: attention(lse=z(2, 5, 2)),
        lambda: rotate(rope=two), lambda: rotate(pos=None), lambda: rotate(q=None, k=None), lambda: rotate(k=k.float()),
        lambda: rotate(q_out=q[:, :4]), lambda: rotate(q=None, q_out=q), lambda: rotate(k=wide[..., 1:65]), lambda: rotate(status=lens),
        lambda: rotate(k=k[:, :1].expand(2, 5, 2, 64)), lambda: rotate(q_out=q[:, :1].expand(2, 5, 4, 64)), lambda: rotate(rope=None),
        lambda: read(units=eight), lambda: read(k_out=back.float()), lambda: read(k_out=back[:, :32]), lambda: read(v_out=back[:2]),
        lambda: read(ids=z(2, dtype=torch.int32)), lambda: read(k_out=z(7, 64, 64, dtype=bf)), lambda: read(ids=[0]),
        lambda: nosa.nosa_rope(z(9, 32)), lambda: nosa.nosa_rope(z(9, 32, 2), axes=[0] * 31), lambda: nosa.nosa_rope(z(9, 32, 2).half()),
        lambda: nosa.nosa_rope(z(32, 9, 2).transpose(0, 1)), lambda: nosa.nosa_rope(z(9, 32, 2).cpu()),
        lambda: rotate(rope=nosa.nosa_rope(z(9, 64, 2))), lambda: rotate(rope=nosa.nosa_rope(z(9, 4, 2))),
        lambda: rotate(rope=nosa.nosa_rope(z(9, 32, 2), axes=[4] * 32), pos=z(5, 2, 5, dtype=torch.int32)),
        lambda: nosa.nosa_rotate(other, rope, pos, q), lambda: nosa.nosa_quant4_read(other, units, back)]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, nosa.NosaError)):
            f()
            print("not refused:", i)
    attention(mass=mass, lse=z(2, 5, 4), rope=rope, positions=pos)  # and what they vary from is accepted
    rotate(rope=two, pos=z(2, 2, 5, dtype=torch.int32))
    rotate()
    read()
    append(rope=rope, positions=pos[None])
    torch.cuda.synchronize()
    assert lens.tolist() == [5] * U and not out.any()
