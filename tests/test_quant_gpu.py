"""The 8-bit block cache on the GPU against the fp64 oracle: append, attention,
eviction, and the three of them as a generation loop.

Tolerances. A scale is one fp32 division (2^-24) of an exact maximum. A code is
e4m3(x * inv) with inv rounded once and the product once, so the number that is
rounded is within 2^-23 + 2^-24 (taken: 2^-22) of the quotient: the code is a
nearest one up to that. Attention: with A the weighted mean of |v| and S the largest
sum |q_x k_x| / sqrt(d) of a row, a logit is off by at most 2^-18 S + 2^-22 |l|: the
tensor cores add d products in at most d / 8 = 16 steps of truncating fp32 additions
(2^-23 each, of partial sums that S bounds), the operands of an fp32 query carry 22
bits, the scaling adds three roundings; weights are then off by twice that
relatively, plus 2^-20 for exp and normalisation and 2^-23 for each of the n / 16
additions. The weights enter the second product with 11 bits (2^-11 of A) where the
output is bf16, with 22 bits where it is fp32; the output's own rounding is half a
step, 2^-8 (bf16) or 2^-24 (fp32).
"""
import os

import numpy as np
import pytest
import torch

import trainable_sparse_attention_decode_gb300 as nosa
from oracle import quant_oracle as Q

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
B = 64
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def dev(x, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(x)).cuda().to(dtype) if dtype else torch.as_tensor(np.ascontiguousarray(x)).cuda()


def f64(t):
    return t.detach().double().cpu().numpy()


def config(batch, hq, hkv, d, dtype):
    return nosa.nosa_config(batch, hq, hkv, d, dtype, 1, 0, 64)


def tail_arrays(cfg, tail, d, dtype):
    """k [U][64][d], v, e [U][64] of tail units, as fp64."""
    t = tail.view(-1, nosa.nosa_payload_bytes(cfg))
    elt = 4 if dtype == "f32" else 2
    kb = B * d * elt
    U = t.shape[0]
    k = t[:, :kb].contiguous().view(DT[dtype]).view(U, d * elt // 16, B, 16 // elt).transpose(1, 2).reshape(U, B, d)
    v = t[:, kb:2 * kb].contiguous().view(DT[dtype]).view(U, B, d)
    return f64(k), f64(v), f64(t[:, 2 * kb:2 * kb + 4 * B].contiguous().view(torch.float32))


def make_tail(cfg, k, v, e, d, dtype):
    """Tail units from k, v [U][64][d] (values of the type), e [U][64]."""
    U, elt = k.shape[0], 4 if dtype == "f32" else 2
    c = 16 // elt
    t = torch.zeros(U, nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    kb = B * d * elt
    t[:, :kb] = dev(k, DT[dtype]).view(U, B, d // c, c).transpose(1, 2).contiguous().view(U, -1).view(torch.uint8)
    t[:, kb:2 * kb] = dev(v, DT[dtype]).contiguous().view(U, -1).view(torch.uint8)
    t[:, 2 * kb:2 * kb + 4 * B] = dev(e.astype(np.float32)).view(torch.uint8)
    return t.view(-1)


class Model:
    """What the cache should hold: every unit's tokens as given (the type's values)."""

    def __init__(self, U, d):
        self.k = [np.zeros((0, d)) for _ in range(U)]
        self.v = [np.zeros((0, d)) for _ in range(U)]
        self.e = [np.zeros(0) for _ in range(U)]

    def add(self, u, k, v, e):
        self.k[u] = np.concatenate([self.k[u], k])
        self.v[u] = np.concatenate([self.v[u], v])
        self.e[u] = np.concatenate([self.e[u], e])


def check_blocks(images, k, v, e, d):
    """Unit images [n] against blocks k, v [n][64][d], e [n][64] (finite)."""
    k8, v8, e8, s = Q.decode(images, d)
    assert np.array_equal(e8, e)
    live = ~np.isneginf(e)[..., None]
    for got, x, sc in ((k8, k, s[:, 0]), (v8, v, s[:, 1])):
        x = np.where(live, x, 0.0)
        want = np.abs(x).max((1, 2)) / 448
        assert np.all(np.abs(sc - want) <= want * 2.0 ** -23)
        y = np.divide(x, want[:, None, None], out=np.zeros_like(x), where=want[:, None, None] > 0)
        assert np.all(np.abs(got - y) <= Q.nearest_distance(y) + np.abs(y) * 2.0 ** -21)
    assert not images[:, 2 * B * d + 4 * B + 8:].any()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,batch,hq,hkv,d,steps,strided", [
    ("bf16", 2, 8, 2, 128, [1, 62, 1, 1, 64, 130, 3, 1], False),
    ("f32", 1, 4, 1, 64, [63, 1, 65, 200, 1], False),
    ("bf16", 3, 3, 3, 64, [1000, 1, 24, 64], True),
    ("f32", 2, 6, 3, 128, [64, 127, 2, 1, 129], True),
    ("bf16", 1, 8, 1, 128, [1] * 66, False)])
def test_append_matches_oracle(dtype, batch, hq, hkv, d, steps, strided):
    rng = np.random.default_rng(sum(steps) + d)
    U, cap = batch * hkv, sum(steps) // B + 2
    cfg = config(batch, hq, hkv, d, dtype)
    extra = 3
    tab = rng.permutation(U * cap + extra)[:U * cap].reshape(U, cap).astype(np.int32)
    units = torch.full((U * cap + extra, Q.unit_bytes(d)), 0xA5, dtype=torch.uint8, device="cuda")
    tail = torch.full((U * nosa.nosa_payload_bytes(cfg),), 0x5A, dtype=torch.uint8, device="cuda")
    lens = torch.zeros(U, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    model = Model(U, d)
    t_tab = dev(tab)
    for i, n in enumerate(steps):
        wide = torch.randn(batch, n, 2 * hkv + 1, d, device="cuda").mul_(rng.uniform(0.1, 30)).to(DT[dtype])
        k, v = wide[:, :, :hkv], wide[:, :, hkv:2 * hkv]
        if not strided:
            k, v = k.contiguous(), v.contiguous()
        e = rng.normal(size=(batch, n, hkv)).astype(np.float32)
        e[rng.random(size=e.shape) < 0.05] = -np.inf
        if i == 1:
            e[:] = 0.0
        n_new = rng.integers(0, n + 1, size=batch).astype(np.int32) if i % 3 == 2 else None
        before = tail.clone()
        nosa.nosa_quant_append(cfg, k, v, None if i == 1 else dev(e), units, t_tab, tail, lens,
                               n_new=None if n_new is None else dev(n_new), status=status)
        kf, vf = f64(k), f64(v)
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
            check_blocks(images[tab[u, :nf]], cut(model.k[u]), cut(model.v[u]), cut(model.e[u])[..., 0], d)
    assert (images[~used] == 0xA5).all()


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 128)])
@pytest.mark.parametrize("n", [64, 128])
def test_append_special_values(dtype, d, n):
    """Blocks of zeros, all masked, of tiny and of huge numbers, with NaN and infinities in masked
    and in live tokens, lowest logits: n = 64 takes the single launch, 128 the two."""
    cases = ["zeros", "masked", "tiny", "huge", "nan masked", "nan live", "inf live", "lowest", "one token"]
    rng = np.random.default_rng(5)
    U = len(cases)
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
    x[5, 7, 0, 3] = np.nan
    x[6, 63, 0, d - 1] = -np.inf
    e[7] = low
    e[8] = -np.inf
    e[8, 17] = 2.0
    cfg = config(U, 1, 1, d, dtype)
    nb = n // B
    units = torch.empty(U * nb, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
    tab = dev(np.arange(U * nb).reshape(U, nb).astype(np.int32))
    tail = torch.zeros(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(U, dtype=torch.int32, device="cuda")
    kt, vt = dev(x, DT[dtype]), dev(v, DT[dtype])
    nosa.nosa_quant_append(cfg, kt, vt, dev(e), units, tab, tail, lens)
    img = units.cpu().numpy().reshape(U, nb, -1)
    kf, vf = f64(kt)[:, :, 0].reshape(U, nb, B, d), f64(vt)[:, :, 0].reshape(U, nb, B, d)
    ef = e[:, :, 0].reshape(U, nb, B)
    for u, name in enumerate(cases):
        k8, v8, e8, s = Q.decode(img[u], d)
        if name in ("nan live", "inf live"):
            bad = ~np.isfinite(kf[u]).all((1, 2))
            assert np.array_equal(np.isnan(s[:, 0]), bad) and not k8[bad].any()
            keep = ~bad
            check_blocks(img[u][keep], kf[u][keep], vf[u][keep], ef[u][keep].astype(np.float64), d)
        elif name == "tiny":
            assert not s[:, 0].any() and not k8.any() and s[:, 1].all()
        elif name in ("zeros", "masked"):
            assert not s[:, 0].any() and not k8.any()
            assert np.array_equal(e8, ef[u].astype(np.float64))
        else:
            kk = np.where(np.isfinite(kf[u]), kf[u], 0.0)  # only masked tokens hold them here
            check_blocks(img[u], kk, vf[u], ef[u].astype(np.float64), d)


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
    nosa.nosa_quant_append(cfg, k, k, None, units, dev(tab), tail, lens, status=status)
    fits = n == 2
    assert lens.tolist() == [lens0[0], lens0[1], lens0[2], 60 + (n if fits else 0)]
    assert status.item() == nosa.NOSA_QUANT_INDEX | nosa.NOSA_QUANT_CAPACITY
    assert (units == 7).all()
    t = tail.view(U, -1)
    assert (t[:3] == 9).all() and bool((t[3] == 9).all()) == (not fits)


def test_append_bad_entries_and_counts():
    """Destinations outside the pool are skipped and flagged, counts clamped and flagged."""
    cfg = config(3, 1, 1, 64, "f32")
    units = torch.full((2, Q.unit_bytes(64)), 3, dtype=torch.uint8, device="cuda")
    tab = dev(np.array([[2, 1], [-1, 0], [0, 0]], np.int32))
    tail = torch.zeros(3 * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    lens, status = torch.zeros(3, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    k = torch.randn(3, 70, 1, 64, device="cuda")
    out = torch.empty_like(lens)
    nosa.nosa_quant_append(cfg, k, k, None, units, tab, tail, lens, lens_out=out, status=status,
                           n_new=dev(np.array([70, 99, -5], np.int32)))
    assert out.tolist() == [70, 70, 0] and lens.tolist() == [0, 0, 0]
    assert (units == 3).all() and status.item() == nosa.NOSA_QUANT_INDEX


def test_append_nothing():
    cfg = config(2, 2, 2, 64, "bf16")
    lens = dev(np.array([3, 64, 0, 70], np.int32))
    out = torch.zeros_like(lens)
    units = torch.zeros(4, Q.unit_bytes(64), dtype=torch.uint8, device="cuda")
    tail = torch.zeros(4 * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    k = torch.zeros(2, 0, 2, 64, dtype=torch.bfloat16, device="cuda")
    nosa.nosa_quant_append(cfg, k, k, None, units, dev(np.zeros((4, 2), np.int32)), tail, lens, lens_out=out)
    assert out.tolist() == [3, 64, 0, 70]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
class Cache:
    """A cache with random contents: device arrays and their values."""

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
        k = (rng.normal(size=(pool, 1, d)) + rng.normal(size=(pool, B, d)) * 0.5) * scale
        v = rng.normal(size=(pool, B, d))
        e = rng.normal(size=(pool, B))
        e[rng.random(size=e.shape) < masked] = -np.inf
        self.images = Q.encode(k, v, e)
        self.tk = f64(torch.as_tensor(rng.normal(size=(U, B, d)) * scale).to(DT[dtype]))
        self.tv = f64(torch.as_tensor(rng.normal(size=(U, B, d))).to(DT[dtype]))
        self.te = rng.normal(size=(U, B)).astype(np.float32)
        self.te[rng.random(size=self.te.shape) < masked] = -np.inf

    def upload(self):
        dtype, _, _, _, d = self.dims
        self.units, self.t_tab, self.t_lens = dev(self.images), dev(self.tab), dev(self.lens)
        self.tail = make_tail(self.cfg, self.tk, self.tv, self.te, d, dtype)
        return self

    def tokens(self, u):
        """K, V, e of unit u's tokens in fp64 (skipped entries: masked)."""
        nf, nt = divmod(int(self.lens[u]), B)
        d = self.dims[4]
        ids = self.tab[u, :nf]
        ok = (ids >= 0) & (ids < len(self.images))
        k8, v8, e, s = Q.decode(self.images[np.where(ok, ids, 0)], d)
        e = np.where(ok[:, None], e, -np.inf)
        K = np.concatenate([(k8 * s[:, 0, None, None]).reshape(-1, d), self.tk[u, :nt]])
        V = np.concatenate([(v8 * s[:, 1, None, None]).reshape(-1, d), self.tv[u, :nt]])
        return K, V, np.concatenate([e.ravel(), self.te[u, :nt].astype(np.float64)])

    def run(self, q, q_len=None, mass=None, decay=1.0, **kw):
        out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        lse = torch.full(q.shape[:3], 7.0, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.workspace = nosa.nosa_quant_attention(
            self.cfg, self.units, self.t_tab, self.tail, self.t_lens, q, out, lse=lse, mass=mass, decay=decay,
            q_len=None if q_len is None else dev(np.asarray(q_len, np.int32)), status=status, **kw)
        return out, lse, status.item()

    def check(self, q, out, lse, q_len=None, mass0=None, mass=None, decay=1.0):
        dtype, batch, hq, hkv, d = self.dims
        T, G = q.shape[1], hq // hkv
        qf, of, lf = f64(q), f64(out), f64(lse)
        p_bits, o_bits = (2.0 ** -11, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -21, 2.0 ** -24)
        for u in range(batch * hkv):
            b, h = divmod(u, hkv)
            n, tq = int(self.lens[u]), T if q_len is None else q_len[b]
            K, V, e = self.tokens(u)
            rows = qf[b, :tq, h * G:(h + 1) * G].reshape(tq * G, d)
            sees = np.repeat(n - tq + 1 + np.arange(tq), G)
            want, wl, w, A, S = Q.attend(rows, K, V, e, sees)
            got = of[b, :tq, h * G:(h + 1) * G].reshape(tq * G, d)
            gl = lf[b, :tq, h * G:(h + 1) * G].reshape(-1)
            empty = np.isneginf(wl)
            assert np.array_equal(np.isneginf(gl), empty), u
            assert not got[empty].any()
            dl = 2.0 ** -18 * S + 2.0 ** -22 * np.abs(np.where(empty, 0.0, wl))
            rel = 2 * dl + 2.0 ** -20 + (n / 16 + 16) * 2.0 ** -23
            tol = o_bits * np.abs(want) + (p_bits + 2 * rel[:, None]) * A + 1e-30
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


def query(rng, batch, T, hq, d, dtype, scale=1.5):
    return dev(rng.normal(size=(batch, T, hq, d)) * scale, DT[dtype])


CASES = [  # dtype, batch, hq, hkv, d, lens by request (heads differ by -h), queries
    ("bf16", 2, 8, 2, 128, [700, 64], 1), ("f32", 1, 4, 1, 64, [2031], 1), ("bf16", 3, 3, 3, 64, [1, 63, 65], 1),
    ("f32", 2, 12, 4, 128, [130, 127], 1), ("bf16", 1, 12, 2, 128, [1300], 1), ("bf16", 1, 8, 1, 64, [4000], 1),
    ("f32", 1, 2, 2, 128, [0], 1), ("bf16", 2, 8, 2, 128, [700, 3], 8), ("f32", 1, 6, 2, 64, [333], 5),
    ("bf16", 1, 8, 1, 128, [640], 32), ("f32", 1, 8, 1, 128, [200], 17), ("bf16", 1, 4, 4, 64, [129], 128),
    ("bf16", 40, 4, 4, 64, [70 + 5 * i for i in range(40)], 1), ("bf16", 2, 6, 1, 128, [190, 64], 3),
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


@pytest.mark.parametrize("dtype,hq,hkv,d,T", [
    ("bf16", 6, 3, 128, 1), ("bf16", 6, 3, 64, 1), ("f32", 6, 3, 128, 1), ("f32", 6, 3, 64, 1), ("bf16", 8, 2, 128, 4),
    ("bf16", 8, 2, 64, 4), ("bf16", 8, 2, 128, 8), ("f32", 8, 2, 64, 8), ("f32", 8, 2, 128, 7)])
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
    _, _, status = c.run(q, q_len=[6, 7, -1, 6])  # counts out of range are clamped and flagged
    assert status == nosa.NOSA_QUANT_INDEX


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 9])
def test_attention_masks(dtype, T):
    """Units with every token masked, with only the tail or only one block visible, with lowest
    logits everywhere, with NaN keys and values in masked places, with a block whose scale is NaN."""
    rng = np.random.default_rng(21)
    hq, d = 8, 64
    names = ["all masked", "tail only", "one block", "lowest", "nan masked", "block masked", "lowest but one"]
    U = len(names)
    c = Cache(rng, dtype, U, hq, 1, d, [300] * U, masked=0.0)
    low = np.finfo(np.float32).min

    def logits(u, j, val):
        at = 2 * B * d
        e = c.images[c.tab[u, j], at:at + 4 * B].view(np.float32)
        e[:] = val

    for j in range(4):
        for u in (0, 1, 2):
            if not (u == 2 and j == 2):
                logits(u, j, -np.inf)
        for u in (3, 6):
            logits(u, j, low)
    logits(6, 1, np.where(np.arange(B) == 5, 0.5, low))
    c.te[0] = c.te[2] = -np.inf
    c.te[3] = c.te[6] = low
    c.te[4, 3:8] = -np.inf
    c.tk[4, 3:5] = np.nan
    c.tv[4, 4:8] = np.inf
    scales = c.images[c.tab[5, 1], 2 * B * d + 4 * B:2 * B * d + 4 * B + 8].view(np.float32)
    scales[:] = np.nan
    logits(5, 1, -np.inf)
    c.upload()
    q = query(rng, U, T, hq, d, dtype)
    m0 = np.zeros(c.tab.shape, np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass)
    assert status == 0
    with np.errstate(invalid="ignore"):
        c_tk, c_tv = c.tk.copy(), c.tv.copy()
        c.tk[4, 3:8], c.tv[4, 3:8] = 0.0, 0.0  # masked: not looked at
        img = c.images.copy()
        scales[:] = 1.0
        c.check(q, out, lse, mass0=m0, mass=f64(mass))
        c.tk, c.tv, c.images = c_tk, c_tv, img


def test_attention_nan_reaches_only_its_rows():
    """A live NaN (scale) makes the rows that see it NaN and no others; a NaN query its own row."""
    rng = np.random.default_rng(2)
    c = Cache(rng, "bf16", 3, 4, 1, 64, [200, 200, 200])
    c.images[c.tab[1, 1], 2 * B * 64 + 4 * B:2 * B * 64 + 4 * B + 4].view(np.float32)[:] = np.nan  # keys
    c.upload()
    q = query(rng, 3, 1, 4, 64, "bf16")
    q[2, 0, 1, 5] = float("nan")
    out, lse, status = c.run(q)
    assert status == 0
    assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all()
    assert not torch.isnan(out[0]).any() and not torch.isnan(lse[0]).any()
    assert torch.isnan(out[2, 0, 1]).all() and not torch.isnan(out[2, 0, [0, 2, 3]]).any()


def test_attention_value_nan_behind_the_rows_view():
    """Two queries; the newest token's block holds NaN values, and the first query does not see it."""
    rng = np.random.default_rng(4)
    c = Cache(rng, "bf16", 1, 2, 1, 128, [129], masked=0.0)
    c.tv[0, 0] = np.nan
    c.upload()
    q = query(rng, 1, 2, 2, 128, "bf16")
    out, _, _ = c.run(q)
    assert not torch.isnan(out[0, 0]).any() and torch.isnan(out[0, 1]).all()


def test_attention_large_and_small_queries():
    """Queries near the ends of the bf16 range: logits stay what they are."""
    rng = np.random.default_rng(6)
    c = Cache(rng, "bf16", 1, 4, 1, 64, [150], scale=2.0 ** -60).upload()
    q = query(rng, 1, 1, 4, 64, "bf16")
    q[:, :, 0] *= 2.0 ** 60
    q[:, :, 1] *= 2.0 ** -100
    q[:, :, 2] *= 2.0 ** 59
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


def test_attention_units_past_four_gib():
    """Table entries whose byte offset passes 2^32."""
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
    # and the append there
    cfg = c.cfg
    lens = dev(np.array([0], np.int32))
    tail = torch.zeros(nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    k = torch.randn(1, 64, 1, d, device="cuda").bfloat16()
    nosa.nosa_quant_append(cfg, k, k, None, pool, dev(np.array([[n - 2]], np.int32)), tail, lens)
    check_blocks(pool[n - 2:n - 1].cpu().numpy(), f64(k)[:, :, 0], f64(k)[:, :, 0], np.zeros((1, 64)), d)


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


def test_attention_captured_behind_other_work():
    """A capture in which the call follows a fork, a join, a copy and a memset."""
    rng = np.random.default_rng(15)
    c = Cache(rng, "bf16", 2, 8, 2, 64, [900, 65, 300, 128]).upload()
    q = query(rng, 2, 1, 8, 64, "bf16")
    q_in, out, lse = torch.zeros_like(q), torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    mass = torch.zeros(c.tab.shape, device="cuda")
    ws = torch.empty(nosa.nosa_quant_attention_workspace_bytes(c.cfg, c.cap, 1, True), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            q_in.copy_(q)
        mass.zero_()
        main.wait_stream(side)
        nosa.nosa_quant_attention(c.cfg, c.units, c.t_tab, c.tail, c.t_lens, q_in, out, lse=lse, mass=mass, workspace=ws)
        other = out.clone()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            nosa.nosa_quant_attention(c.cfg, c.units, c.t_tab, c.tail, c.t_lens, q_in, out, lse=lse, mass=mass, workspace=ws)
        main.wait_stream(side)
    for _ in range(3):
        q.copy_(query(rng, 2, 1, 8, 64, "bf16"))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        m = f64(mass)  # two calls' weights
        c.check(q, out, lse, mass0=m / 2, mass=m, decay=1.0)
        assert torch.equal(other, out)


def test_first_calls_inside_a_capture():
    """A process whose first calls are captured."""
    import subprocess
    import sys
    code = """
import sys
sys.path[:0] = [%r, %r]
import numpy as np, torch
import test_quant_gpu as t
nosa = t.nosa
rng = np.random.default_rng(3)
c = t.Cache(rng, "f32", 1, 4, 2, 64, [300, 100], cap=6).upload()
q = t.query(rng, 1, 4, 4, 64, "f32")
out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
mass = torch.zeros(c.tab.shape, device="cuda")
k = t.query(rng, 1, 70, 2, 64, "f32")
ws = torch.empty(nosa.nosa_quant_attention_workspace_bytes(c.cfg, c.cap, 4, True), dtype=torch.uint8, device="cuda")
c.t_tab[:, 2:] = torch.arange(4, dtype=torch.int32, device="cuda") + len(c.images)
units = torch.zeros(len(c.images) + 4, c.images.shape[1], dtype=torch.uint8, device="cuda")
units[:len(c.images)] = c.units
c.t_tab[0, :4] = t.dev(c.tab[0, :4])
c.t_tab[1, 1] = len(c.images)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
lens = c.t_lens.clone()
with torch.cuda.graph(g):
    nosa.nosa_quant_attention(c.cfg, units, c.t_tab, c.tail, lens, q, out, lse=lse, mass=mass, workspace=ws)
    nosa.nosa_quant_append(c.cfg, k[:, :, :2], k[:, :, :2], None, units, c.t_tab, c.tail, lens)
    nosa.nosa_quant_evict(c.cfg, 2, 1, c.t_tab, mass, lens)
g.replay()
torch.cuda.synchronize()
c.check(q, out, lse)
assert lens.tolist() == [64 * 2 + (300 + 70) %% 64, 64 * 2 + (100 + 70) %% 64], lens.tolist()
print("ok")
""" % (ROOT, os.path.join(ROOT, "tests"))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("U,cap,budget,recent,kind", [
    (3, 5, 2, 1, "few"), (6, 130, 128, 8, "few"), (4, 1030, 64, 8, "few"), (2, 2000, 1, 0, "ties"), (3, 300, 17, 17, "any"),
    (5, 64, 63, 0, "any"), (2, 700, 350, 3, "nan"), (2, 9000, 4000, 100, "any"), (1, 16384, 5, 2, "ties")])
@pytest.mark.parametrize("in_place", [False, True])
def test_evict_matches_oracle(U, cap, budget, recent, kind, in_place):
    rng = np.random.default_rng(cap + budget)
    mass = {"few": lambda: rng.exponential(size=(U, cap)).round(1), "ties": lambda: np.full((U, cap), 0.25),
            "any": lambda: rng.normal(size=(U, cap)) * 1e3,
            "nan": lambda: np.where(rng.random((U, cap)) < 0.3, np.nan, rng.normal(size=(U, cap)))}[kind]().astype(np.float32)
    if kind == "any":
        mass[:, ::7] = np.inf
        mass[:, 1::9] = -np.inf
    lens = rng.integers(0, cap * B + 1, size=U).astype(np.int32)
    lens[0] = cap * B  # a full row without a tail
    if U > 1:
        lens[1] = budget * B + 63 if budget < cap else cap * B
    tab = np.stack([rng.permutation(cap) for _ in range(U)]).astype(np.int32)
    cfg = config(U, 1, 1, 64, "bf16")
    t, m, n = dev(tab), dev(mass), dev(lens)
    order = torch.full_like(t, -5)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    outs = (None, None, None) if in_place else (torch.full_like(t, -9), torch.full_like(m, -9.0), torch.full_like(n, -9))
    nosa.nosa_quant_evict(cfg, budget, recent, t, m, n, *outs, order=order, status=status)
    got = (t, m, n) if in_place else outs
    if not in_place:
        assert np.array_equal(t.cpu().numpy(), tab) and np.array_equal(m.cpu().numpy(), mass, equal_nan=True)
    assert status.item() == 0
    for u in range(U):
        wt, wm, wn, wo = Q.evict(tab[u], mass[u], int(lens[u]), budget, recent)
        assert got[2][u].item() == wn
        assert np.array_equal(got[0][u].cpu().numpy(), wt), u
        assert np.array_equal(order[u].cpu().numpy(), wo), u
        assert np.array_equal(got[1][u].cpu().numpy(), wm, equal_nan=True), u


def test_evict_leaves_units_with_bad_lengths():
    cfg = config(2, 1, 1, 64, "bf16")
    tab = dev(np.arange(8).reshape(2, 4).astype(np.int32))
    mass = dev(np.arange(8).reshape(2, 4).astype(np.float32))
    lens = dev(np.array([-1, 4 * B + 1], np.int32))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    nosa.nosa_quant_evict(cfg, 1, 0, tab, mass, lens, status=status)
    assert status.item() == nosa.NOSA_QUANT_INDEX and lens.tolist() == [-1, 257]
    assert tab.flatten().tolist() == list(range(8)) and mass.flatten().tolist() == list(range(8))


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,batch,hq,hkv,d", [("bf16", 2, 8, 2, 128), ("f32", 1, 4, 2, 64)])
def test_generation_loop_in_a_graph(dtype, batch, hq, hkv, d):
    """Prompt, observation, first eviction, then a captured step (append, attention, eviction)
    replayed past several block ends: outputs, weights, lengths and order against a model that
    keeps every token in fp64; two graphs share the workspace."""
    rng = np.random.default_rng(d)
    U, G = batch * hkv, hq // hkv
    budget, recent, cap, decay = 4, 1, 9, 0.9
    cfg = config(batch, hq, hkv, d, dtype)
    units = torch.zeros(U * cap, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
    tab = dev(rng.permutation(U * cap).reshape(U, cap).astype(np.int32))
    tail = torch.zeros(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
    lens = torch.zeros(U, dtype=torch.int32, device="cuda")
    mass = torch.zeros(U, cap, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    model = Model(U, d)
    weight = [np.zeros(cap, np.float64) for _ in range(U)]

    def tokens(n):
        k, v = (query(rng, batch, n, hkv, d, dtype, 1.0) for _ in range(2))
        return k, v, dev(rng.normal(size=(batch, n, hkv)).astype(np.float32))

    def model_append(k, v, e):
        for u in range(U):
            b, h = divmod(u, hkv)
            model.add(u, f64(k)[b, :, h], f64(v)[b, :, h], f64(e)[b, :, h])

    def model_attend(q, out, lse):
        """Checks a call against the cache's own stored values and updates the weights."""
        T = q.shape[1]
        c = Cache.__new__(Cache)
        c.dims, c.cfg, c.cap = (dtype, batch, hq, hkv, d), cfg, cap
        c.images, c.tab, c.lens = units.cpu().numpy(), tab.cpu().numpy(), lens.cpu().numpy()
        c.tk, c.tv, te = tail_arrays(cfg, tail, d, dtype)
        c.te = te.astype(np.float32)
        m0 = np.stack(weight).astype(np.float32)
        got = f64(mass)
        c.check(q, out, lse, mass0=m0, mass=got, decay=decay)
        for u in range(U):  # what is stored is what was appended, rounded
            n = int(c.lens[u])
            assert n == len(model.e[u])
            K, V, e = c.tokens(u)
            assert np.array_equal(e, model.e[u])
            # e4m3: half a step is 2^-4 of the value or 2^-10 of the scale (max / 448)
            for x, y in ((K, model.k[u]), (V, model.v[u])):
                assert np.all(np.abs(x - y) <= np.abs(y) * 2.0 ** -4 + 2.0 ** -10 * np.abs(y).max() / 448 + 1e-9)
            weight[u] = got[u].copy()
        assert status.item() == 0

    def model_evict():
        for u in range(U):
            n = len(model.e[u])
            _, wm, wn, order = Q.evict(np.arange(cap), weight[u].astype(np.float32), n, budget, recent)
            nf, kept = n // B, wn // B
            take = np.concatenate([np.arange(B) + B * j for j in order[:kept]] + [np.arange(nf * B, n)]).astype(int)
            model.k[u], model.v[u], model.e[u] = model.k[u][take], model.v[u][take], model.e[u][take]
            weight[u] = wm.astype(np.float64)
            assert lens[u].item() == wn

    # the prompt, its last 8 tokens' look back, the first eviction
    k, v, e = tokens(8 * B + 21)
    nosa.nosa_quant_append(cfg, k, v, e, units, tab, tail, lens, status=status)
    model_append(k, v, e)
    q = query(rng, batch, 8, hq, d, dtype)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    nosa.nosa_quant_attention(cfg, units, tab, tail, lens, q, out, lse=lse, mass=mass, decay=decay, status=status)
    model_attend(q, out, lse)
    nosa.nosa_quant_evict(cfg, budget, recent, tab, mass, lens, status=status)
    model_evict()

    # one step, captured twice on a stream of its own; the graphs alternate and share the workspace
    ws = torch.empty(nosa.nosa_quant_attention_workspace_bytes(cfg, cap, 1, True), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    bufs, graphs = [], []
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        k, v, e = tokens(1)
        q = query(rng, batch, 1, hq, d, dtype)
        out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=stream):
            nosa.nosa_quant_append(cfg, k, v, e, units, tab, tail, lens, status=status)
            nosa.nosa_quant_attention(cfg, units, tab, tail, lens, q, out, lse=lse, mass=mass, decay=decay,
                                      workspace=ws, status=status)
        bufs.append((k, v, e, q, out, lse))
        graphs.append(g)
    evict = torch.cuda.CUDAGraph()
    with torch.cuda.graph(evict, stream=stream):
        nosa.nosa_quant_evict(cfg, budget, recent, tab, mass, lens, status=status)
    for step in range(3 * B):
        k, v, e, q, out, lse = bufs[step % 2]
        for dst, src in zip((k, v, e), tokens(1)):
            dst.copy_(src)
        q.copy_(query(rng, batch, 1, hq, d, dtype))
        graphs[step % 2].replay()
        model_append(k, v, e)
        if step % 5 == 0 or len(model.e[0]) % B in (0, 1, 63):
            torch.cuda.synchronize()
            model_attend(q, out, lse)
        else:
            got = f64(mass)
            for u in range(U):
                weight[u] = got[u].copy()
        evict.replay()
        model_evict()
    assert status.item() == 0


def test_tensors_elsewhere_are_refused():
    cfg = config(1, 2, 1, 64, "bf16")
    cfg.device = 1  # the tensors are on device 0
    lens = torch.zeros(1, dtype=torch.int32, device="cuda:0")
    units = torch.zeros(1, Q.unit_bytes(64), dtype=torch.uint8, device="cuda:0")
    tab = torch.zeros(1, 1, dtype=torch.int32, device="cuda:0")
    with pytest.raises(ValueError, match="device"):
        nosa.nosa_quant_evict(cfg, 1, 0, tab, torch.zeros(1, 1, device="cuda:0"), lens)
    tail = torch.zeros(nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda:0")
    q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16, device="cuda:0")
    with pytest.raises(ValueError, match="device"):
        nosa.nosa_quant_attention(cfg, units, tab, tail, lens, q, torch.empty_like(q))
    with pytest.raises(ValueError, match="device"):
        nosa.nosa_quant_append(cfg, q[:, :, :1], q[:, :, :1], None, units, tab, tail, lens)


def test_binding_refusals():
    """Wrong types, shapes, strides, sizes and alignments are refused before anything runs."""
    cfg = config(2, 4, 2, 64, "bf16")
    U, cap, bf = 4, 3, torch.bfloat16
    z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    units, tab = z(6, Q.unit_bytes(64), dtype=torch.uint8), z(U, cap, dtype=torch.int32)
    tail, lens = z(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8), z(U, dtype=torch.int32)
    k, q, mass = z(2, 5, 2, 64, dtype=bf), z(2, 5, 4, 64, dtype=bf), z(U, cap)
    out = torch.empty_like(q)
    ws = z(nosa.nosa_quant_attention_workspace_bytes(cfg, cap, 5, True), dtype=torch.uint8)

    def append(k=k, v=k, e=None, units=units, tab=tab, tail=tail, lens=lens, **kw):
        nosa.nosa_quant_append(cfg, k, v, e, units, tab, tail, lens, **kw)

    def attention(units=units, tab=tab, tail=tail, lens=lens, q=q, out=out, workspace=ws, **kw):
        nosa.nosa_quant_attention(cfg, units, tab, tail, lens, q, out, workspace=workspace, **kw)

    def evict(tab=tab, mass=mass, lens=lens, budget=2, recent=1, **kw):
        nosa.nosa_quant_evict(cfg, budget, recent, tab, mass, lens, **kw)

    wide = z(2, 5, 2, 72, dtype=bf)
    bad = [
        lambda: append(k=k.float()), lambda: append(k=k[:, :, :1]), lambda: append(v=k[:, :4]),
        lambda: append(k=z(2, 5, 64, 2, dtype=bf).transpose(2, 3)), lambda: append(k=wide[..., 1:65]),
        lambda: append(k=z(2, 5, 2, 68, dtype=bf)[..., :64]), lambda: append(e=z(2, 5, 4)), lambda: append(e=k[..., 0]),
        lambda: append(units=units.view(-1)[1:]), lambda: append(units=units.view(-1)[:100]),
        lambda: append(tail=tail[:-256]), lambda: append(lens=lens[:2]), lambda: append(lens=lens.float()),
        lambda: append(tab=tab.long()), lambda: append(tab=tab[:2]), lambda: append(lens_out=z(U)),
        lambda: append(n_new=z(3, dtype=torch.int32)), lambda: append(status=z(2, dtype=torch.int32)),
        lambda: attention(q=q.float()), lambda: attention(q=z(2, 129, 4, 64, dtype=bf)), lambda: attention(out=out[:, :4]),
        lambda: attention(out=z(2, 5, 8, 64, dtype=bf)[:, :, ::2]), lambda: attention(out=q), lambda: attention(lse=z(2, 5, 2)),
        lambda: attention(mass=z(U, cap + 1)), lambda: attention(mass=mass, decay=2.0), lambda: attention(mass=mass, workspace=ws[:-256]),
        lambda: attention(workspace=ws[16:]), lambda: attention(q_len=z(3, dtype=torch.int32)),
        lambda: attention(tail=tail.float()), lambda: evict(mass=mass.double()), lambda: evict(mass=mass[:, :2]),
        lambda: evict(budget=0, recent=0), lambda: evict(recent=3), lambda: evict(order=z(U, cap)),
        lambda: evict(tab_out=z(U, cap + 1, dtype=torch.int32)), lambda: evict(lens_out=z(U + 1, dtype=torch.int32))]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, nosa.NosaError)):
            f()
            print("not refused:", i)
    attention(mass=mass, lse=z(2, 5, 4))  # and what they vary from is accepted
    append()
    evict()
    torch.cuda.synchronize()
    assert lens.tolist() == [5] * U and not out.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 3, 8])
def test_attention_masked_codes(dtype, d, T):
    """Masked tokens of a block hold the codes that are no numbers: one token, several of every slice,
    and all of a block contribute nothing. 4, 12 and 32 rows take every shape of tile."""
    rng = np.random.default_rng(31 + T)
    c = Cache(rng, dtype, 3, 4, 1, d, [64 * 5 + 9, 64 * 3, 64 * 40 + 1], masked=0.0)
    ko, vo = Q.code_offsets(d)
    gone = {c.tab[0, 1]: [17], c.tab[0, 4]: [0, 5, 10, 15, 18, 35, 52, 63], c.tab[1, 0]: list(range(B)),
            c.tab[1, 2]: list(range(1, B)), c.tab[2, 39]: [62, 63]}
    for i, tokens in gone.items():
        c.images[i, 2 * B * d:2 * B * d + 4 * B].view(np.float32)[tokens] = -np.inf
        for n, t in enumerate(tokens):
            c.images[i, vo[t]] = 0x7F if n % 2 else 0xFF
            c.images[i, ko[t]] = 0xFF if n % 3 else 0x7F
    c.upload()
    q = query(rng, 3, T, 4, d, dtype)
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    for _ in range(2):
        mass = dev(m0)
        out, lse, status = c.run(q, mass=mass)
        assert status == 0
        c.check(q, out, lse, mass0=m0, mass=f64(mass))
    assert torch.equal(c.units, dev(c.images))  # the cache itself keeps its bytes


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,T", [(4, 2), (1, 70)])
def test_attention_codes_that_are_no_numbers(dtype, hq, T):
    """A value code that is no number in a token that is not masked reaches the rows that see that token,
    in its dim, and no others."""
    rng = np.random.default_rng(33)
    d, n = 64, 192
    c = Cache(rng, dtype, 1, hq, 1, d, [n], masked=0.0)
    _, vo = Q.code_offsets(d)
    last = c.tab[0, 2]
    if T == 2:  # the first query sees masked tokens of the last block only
        c.images[last, 2 * B * d:2 * B * d + 4 * B].view(np.float32)[:63] = -np.inf
    c.images[last, vo[63, 7]] = 0x7F
    c.upload()
    q = query(rng, 1, T, hq, d, dtype)
    out, lse, status = c.run(q)
    assert status == 0 and not torch.isnan(lse).any()
    sees = n - T + 1 + np.arange(T)
    reached = sees == n
    nan = torch.isnan(out[0]).cpu().numpy()  # [T][hq][d]
    assert nan[reached][:, :, 7].all() and not nan[~reached].any() and not np.delete(nan, 7, axis=2).any()
    K, V, e = c.tokens(0)
    for t in np.flatnonzero(~reached):  # and those rows are right
        want, wl, _, A, S = Q.attend(f64(q)[0, t], K, np.nan_to_num(V), e, np.full(hq, sees[t]))
        assert np.all(np.abs(f64(out)[0, t] - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2.0 ** -16 * S[:, None]) * A)
        assert np.all(np.abs(f64(lse)[0, t] - wl) <= 2.0 ** -18 * S + 2.0 ** -18 * (1 + np.abs(wl)))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T", [1, 3, 8])
@pytest.mark.parametrize("outlier", [300.0, 30000.0])
def test_attention_queries_with_an_outlier(dtype, d, T, outlier):
    """One element of a query is far larger than the others and meets keys of zero: the others keep
    their bits. An element is held to 2^-22 of itself (bf16: exactly) or to 2^-39 of the row's largest,
    which for an outlier of 2^15 is 2^-24: summed over 128 dims of keys of about 1, over sqrt(d), below
    2^-20, a hundredth of the 2^-18 S (S about 10) that the check allows a logit."""
    rng = np.random.default_rng(41 + d)
    c = Cache(rng, dtype, 2, 4, 1, d, [64 * 4 + 3, 64 * 2], masked=0.0)
    ko, _ = Q.code_offsets(d)
    c.images[:, ko[:, 9]] = 0
    c.tk[:, :, 9] = 0.0
    c.upload()
    q = query(rng, 2, T, 4, d, dtype, scale=1.0)
    q[..., 9] = outlier
    q[:, :, 1, 9] *= -1
    out, lse, status = c.run(q)
    assert status == 0
    c.check(q, out, lse)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top", [-140, -126, -113, -112, -108, -90, 90, 111, 126, 127.9])
def test_attention_queries_at_the_ends_of_the_range(dtype, d, top):
    """Rows whose largest element is 2^top, with keys that bring the logits back to about 1 where a
    block can hold them (largest element 2^-99 to 2^120)."""
    rng = np.random.default_rng(43)
    key = 2.0 ** min(max(-top, -100.0), 118.0)
    c = Cache(rng, dtype, 1, 4, 1, d, [64 * 3 + 5], masked=0.0)
    k = rng.normal(size=(len(c.images), B, d)).clip(-3, 3) * key
    _, v8, e, s = Q.decode(c.images, d)
    c.images = Q.encode(k, v8 * s[:, 1, None, None], e)
    c.tk = f64(torch.as_tensor(rng.normal(size=c.tk.shape).clip(-3, 3) * key).to(DT[dtype]))
    c.upload()
    x = rng.uniform(-1, 1, size=(1, 1, 4, d))
    x[..., 3] = 1.0
    q = dev(x * 2.0 ** top, DT[dtype])
    out, lse, status = c.run(q)
    assert status == 0
    c.check(q, out, lse)


@pytest.mark.parametrize("kind", ["stream", "pointer", "default"])
def test_attention_workspace_belongs_to_the_calls_stream(kind):
    """The workspace of a call on another stream is not memory that was freed on the current one while
    work there still uses it."""
    rng = np.random.default_rng(51)
    c = Cache(rng, "bf16", 2, 8, 2, 64, [700, 64, 300, 129]).upload()
    q = query(rng, 2, 1, 8, 64, "bf16")
    need = nosa.nosa_quant_attention_workspace_bytes(c.cfg, c.cap, 1, False)
    side = torch.cuda.Stream()
    out, lse = torch.empty_like(q), torch.empty(q.shape[:3], device="cuda")
    torch.cuda.synchronize()
    current, other = (side, torch.cuda.default_stream()) if kind == "default" else (torch.cuda.current_stream(), side)
    arg = {"stream": other, "pointer": other.cuda_stream, "default": 0}[kind]
    with torch.cuda.stream(current):
        used = torch.empty(need, dtype=torch.uint8, device="cuda")
        for i in range(200):
            used.fill_(i)
        at = used.data_ptr()
        del used
        ws = nosa.nosa_quant_attention(c.cfg, c.units, c.t_tab, c.tail, c.t_lens, q, out, lse=lse, stream=arg)
    assert ws.numel() == need and (ws.data_ptr() + need <= at or at + need <= ws.data_ptr())
    torch.cuda.synchronize()
    c.check(q, out, lse)


@pytest.mark.parametrize("dtype,batch,hq,hkv,d,T,n,cap", [
    ("bf16", 2, 8, 2, 128, 1, 700, 11), ("bf16", 2, 8, 2, 64, 1, 700, 600), ("f32", 3, 4, 1, 64, 1, 400, 7), ("f32", 1, 4, 2, 128, 3, 999, 16),
    ("bf16", 2, 8, 2, 128, 12, 900, 15), ("f32", 2, 8, 2, 64, 8, 300, 5), ("bf16", 300, 4, 4, 64, 1, 130, 3)])
def test_attention_wait_that_gives_up(dtype, batch, hq, hkv, d, T, n, cap, monkeypatch):
    """Waits that give up at once (set on the host): the status says so, the rows that exist are
    NaN (every unit has blocks), the accumulated weights stay, the kernels end, and the next call is right."""
    rng = np.random.default_rng(61)
    c = Cache(rng, dtype, batch, hq, hkv, d, [n - h for _ in range(batch) for h in range(hkv)], cap=cap).upload()
    q = query(rng, batch, T, hq, d, dtype)
    q_len = [T] * (batch - 1) + [max(1, T - 1)]
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    c.run(q, q_len=q_len, mass=dev(m0))
    ws = c.workspace
    monkeypatch.setenv("NOSA_INJECT_FAIL", "wait")
    for _ in range(3):
        out, lse, status = c.run(q, q_len=q_len, mass=mass, decay=0.5, workspace=ws)
        assert status == nosa.NOSA_QUANT_WAIT
        for b in range(batch):
            assert torch.isnan(out[b, :q_len[b]]).all() and torch.isnan(lse[b, :q_len[b]]).all()
            assert (out[b, q_len[b]:] == 7).all() and (lse[b, q_len[b]:] == 7).all()
        assert np.array_equal(mass.cpu().numpy(), m0)
    monkeypatch.delenv("NOSA_INJECT_FAIL")
    out, lse, status = c.run(q, q_len=q_len, mass=mass, decay=0.5, workspace=ws)
    assert status == 0
    c.check(q, out, lse, q_len=q_len, mass0=m0, mass=f64(mass), decay=0.5)


@pytest.mark.parametrize("dtype,batch,hq,hkv,d,cap", [("bf16", 64, 16, 8, 64, 4), ("f32", 40, 8, 8, 128, 4), ("bf16", 160, 24, 8, 128, 200),
                                                      ("f32", 300, 4, 4, 64, 140)])
def test_calls_behind_each_other_read_what_the_last_one_wrote(dtype, batch, hq, hkv, d, cap):
    """Steps of append, attention and eviction over many units, whose lengths share cache lines: queued
    without a pause and with the GPU waited for after every call, the bits are the same."""
    rng = np.random.default_rng(71)
    U = batch * hkv
    cfg = config(batch, hq, hkv, d, dtype)
    steps = 24
    ins = [(query(rng, batch, 1, hkv, d, dtype, 1.0), query(rng, batch, 1, hkv, d, dtype, 1.0), query(rng, batch, 1, hq, d, dtype)) for _ in range(steps)]
    prompt = query(rng, batch, 3 * B, hkv, d, dtype, 1.0)
    n_new = dev(rng.integers(1, 3 * B - 1, size=batch).astype(np.int32))

    def loop(pause):
        done = torch.cuda.synchronize if pause else lambda: None
        units = torch.zeros(U * 4, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
        tab = torch.zeros(U, cap, dtype=torch.int32, device="cuda")
        tab[:, :4] = torch.arange(U * 4, dtype=torch.int32, device="cuda").view(U, 4)
        tail = torch.zeros(U * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8, device="cuda")
        lens, mass = torch.zeros(U, dtype=torch.int32, device="cuda"), torch.zeros(U, cap, device="cuda")
        ws = torch.zeros(nosa.nosa_quant_attention_workspace_bytes(cfg, cap, 1, True), dtype=torch.uint8, device="cuda")
        outs = [(torch.empty_like(ins[0][2]), torch.empty(batch, 1, hq, device="cuda")) for _ in range(steps)]
        torch.cuda.synchronize()
        nosa.nosa_quant_append(cfg, prompt, prompt, None, units, tab, tail, lens, n_new=n_new)
        done()
        for (k, v, q), (out, lse) in zip(ins, outs):
            nosa.nosa_quant_append(cfg, k, v, None, units, tab, tail, lens)
            done()
            nosa.nosa_quant_attention(cfg, units, tab, tail, lens, q, out, lse=lse, mass=mass, decay=0.9, workspace=ws)
            done()
            nosa.nosa_quant_evict(cfg, 2, 1, tab, mass, lens)
            done()
        torch.cuda.synchronize()
        return [x for pair in outs for x in pair] + [mass, lens, tail, units]

    want = loop(True)
    for _ in range(3):
        assert all(torch.equal(x, y) for x, y in zip(want, loop(False)))


@pytest.mark.parametrize("dtype,hq,hkv,d,T,n", [("bf16", 8, 8, 64, 1, 70), ("bf16", 16, 4, 128, 1, 900), ("f32", 8, 2, 64, 4, 300), ("f32", 8, 4, 128, 1, 64)])
def test_attention_queries_written_by_the_call_before(dtype, hq, hkv, d, T, n):
    """Each call's queries are the outputs of the call before it, in two buffers that are written again
    and again: queued without a pause and with one, the bits are the same."""
    rng = np.random.default_rng(73)
    c = Cache(rng, dtype, 20, hq, hkv, d, [n] * (20 * hkv)).upload()
    first = query(rng, 20, T, hq, d, dtype)
    ws = torch.empty(nosa.nosa_quant_attention_workspace_bytes(c.cfg, c.cap, T), dtype=torch.uint8, device="cuda")

    def chain(pause):
        a, b, seen = first.clone(), torch.empty_like(first), []
        for i in range(40):
            nosa.nosa_quant_attention(c.cfg, c.units, c.t_tab, c.tail, c.t_lens, a, b, workspace=ws)
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


def test_first_evictions_of_two_threads():
    """A process in which threads with tables of different widths evict first, at once: the widest table
    is evicted from afterwards."""
    import subprocess
    import sys
    code = """
import sys, threading
sys.path[:0] = [%r, %r]
import numpy as np, torch
import test_quant_gpu as t
nosa = t.nosa
widths = [6000, 16384, 5200, 9000, 12000, 7000, 16000, 5100]
cfg = t.config(1, 1, 1, 64, "bf16")
def arrays(cap):
    rng = np.random.default_rng(cap)
    mass = rng.random((1, cap)).astype(np.float32)
    return mass, t.dev(np.arange(cap, dtype=np.int32)[None]), t.dev(mass), t.dev(np.array([64 * cap], np.int32))
ins = [arrays(cap) for cap in widths]
torch.cuda.synchronize()
gate, bad = threading.Barrier(len(widths)), []
def first(mass, tab, m, n):
    gate.wait()
    try:
        nosa.nosa_quant_evict(cfg, 16, 4, tab, m, n)
    except Exception as e:
        bad.append(e)
threads = [threading.Thread(target=first, args=x) for x in ins]
[x.start() for x in threads]
[x.join() for x in threads]
mass, tab, m, n = arrays(16384)
nosa.nosa_quant_evict(cfg, 16, 4, tab, m, n)
torch.cuda.synchronize()
assert not bad, bad
for (mass, tab, m, n), cap in zip(ins + [(mass, tab, m, n)], widths + [16384]):
    wt, wm, wn, _ = t.Q.evict(np.arange(cap), mass[0], 64 * cap, 16, 4)
    assert n.item() == wn and np.array_equal(tab[0].cpu().numpy(), wt) and np.array_equal(m[0].cpu().numpy(), wm)
print("ok")
""" % (ROOT, os.path.join(ROOT, "tests"))
    for _ in range(3):
        r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
        assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stdout + r.stderr


@pytest.mark.parametrize("bad", [None, 4096, np.zeros((2, 1, 2, 64), np.float32)])
def test_binding_names_what_is_no_tensor(bad):
    cfg = config(2, 4, 2, 64, "bf16")
    z = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device="cuda")  # noqa: E731
    k, q = z(2, 1, 2, 64, dtype=torch.bfloat16), z(2, 1, 4, 64, dtype=torch.bfloat16)
    cache = dict(units=z(6, Q.unit_bytes(64), dtype=torch.uint8), block_tab=z(4, 3, dtype=torch.int32),
                 tail=z(4 * nosa.nosa_payload_bytes(cfg), dtype=torch.uint8), lens=z(4, dtype=torch.int32))
    calls = [(nosa.nosa_quant_append, dict(k=k, v=k, **cache), dict(e=None)),
             (nosa.nosa_quant_attention, dict(q=q, out=torch.empty_like(q), **cache), {}),
             (nosa.nosa_quant_evict, dict(block_tab=cache["block_tab"], mass=z(4, 3), lens=cache["lens"]), dict(budget=2, n_recent=1))]
    for f, tensors, others in calls:
        for name in tensors:
            with pytest.raises(ValueError, match=f"{name} (is required|must)"):
                f(cfg, **{**tensors, name: bad}, **others)
        f(cfg, **tensors, **others)  # and as it should be it runs
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype,batch,hq,hkv,d,lens,T", [
    ("f32", 2, 8, 2, 128, [333, 64], 3), ("f32", 1, 8, 1, 128, [1000], 2), ("f32", 2, 16, 16, 128, [190, 5], 9), ("f32", 1, 6, 2, 128, [700], 5),
    ("bf16", 1, 16, 2, 128, [2000], 5), ("bf16", 1, 6, 1, 64, [300], 8)])
@pytest.mark.parametrize("with_mass", [False, True])
def test_attention_rows_between_the_tiles(dtype, batch, hq, hkv, d, lens, T, with_mass):
    """9 to 16 rows in fp32 with d = 128, and row counts just above a tile."""
    rng = np.random.default_rng(81)
    c = Cache(rng, dtype, batch, hq, hkv, d, [max(0, n - h) for n in lens for h in range(hkv)]).upload()
    q = query(rng, batch, T, hq, d, dtype)
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0) if with_mass else None
    out, lse, status = c.run(q, mass=mass, decay=0.5)
    assert status == 0
    c.check(q, out, lse, mass0=m0, mass=f64(mass) if with_mass else None, decay=0.5)


@pytest.mark.parametrize("hq,T", [(4, 7), (8, 3)])
def test_attention_long_rings_fp32_16_rows(hq, T):
    rng = np.random.default_rng(83)
    hkv, d = 2, 128
    c = Cache(rng, "f32", 2, hq, hkv, d, [64 * 50] * 4)
    c.lens = np.array([64 * 1300 + 9, 64 * 700, 64 * 2000 + 63, 40], np.int32)
    c.cap = 2001
    c.tab = rng.integers(0, len(c.images), size=(4, c.cap)).astype(np.int32)
    c.upload()
    q = query(rng, 2, T, hq, d, "f32")
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, mass=mass, decay=0.5)
    assert status == 0
    c.check(q, out, lse, mass0=m0, mass=f64(mass), decay=0.5)
    for _ in range(5):
        m1 = dev(m0)
        again = c.run(q, mass=m1, decay=0.5, workspace=c.workspace)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1]) and torch.equal(mass, m1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,q_len", [(12, [12, 1, 0, 5]), (9, [2, 4, 9, 8]), (33, [1, 33, 0, 17])])
def test_attention_tiles_without_rows(dtype, T, q_len):
    """Several tiles of rows, of which a request's queries fill some or none."""
    rng = np.random.default_rng(85)
    c = Cache(rng, dtype, 4, 8, 1, 64, [500, 129, 70, 64]).upload()
    q = query(rng, 4, T, 8, 64, dtype)
    m0 = rng.random(size=c.tab.shape).astype(np.float32)
    mass = dev(m0)
    out, lse, status = c.run(q, q_len=q_len, mass=mass, decay=0.75)
    assert status == 0
    c.check(q, out, lse, q_len=q_len, mass0=m0, mass=f64(mass), decay=0.75)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_strides_of_zero(dtype):
    """Queries, keys and values that are the same for all requests, tokens or heads."""
    rng = np.random.default_rng(87)
    batch, hq, hkv, d, T = 3, 4, 2, 64, 5
    c = Cache(rng, dtype, batch, hq, hkv, d, [200, 65, 128, 7, 300, 64]).upload()
    for shape in ((1, T, hq, d), (batch, 1, hq, d), (batch, T, 1, d), (1, 1, 1, d)):
        q = dev(rng.normal(size=shape), DT[dtype]).expand(batch, T, hq, d)
        out = torch.empty(batch, T, hq, d, dtype=DT[dtype], device="cuda")
        lse = torch.empty(batch, T, hq, device="cuda")
        nosa.nosa_quant_attention(c.cfg, c.units, c.t_tab, c.tail, c.t_lens, q, out, lse=lse)
        c.check(q, out, lse)
    for n in (9, 66):
        for shape in ((1, n, hkv, d), (batch, 1, hkv, d), (batch, n, 1, d)):
            k = dev(rng.normal(size=shape), DT[dtype]).expand(batch, n, hkv, d)
            res = []
            for x in (k, k.contiguous()):
                units = torch.zeros(12, Q.unit_bytes(d), dtype=torch.uint8, device="cuda")
                tail = torch.zeros(6 * nosa.nosa_payload_bytes(c.cfg), dtype=torch.uint8, device="cuda")
                lens = torch.full((6,), 60, dtype=torch.int32, device="cuda")
                nosa.nosa_quant_append(c.cfg, x, x, None, units, dev(np.arange(12).reshape(6, 2)[:, ::-1].astype(np.int32)), tail, lens)
                res.append((units, tail, lens))
            assert all(torch.equal(x, y) for x, y in zip(*res)) and res[0][2].tolist() == [60 + n] * 6


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("f32", 128)])
def test_attention_the_longest_table(dtype, d):
    """16384 blocks and no tail: one block named by every entry, so that the output is the block's and
    every entry weighs the same."""
    rng = np.random.default_rng(89)
    cap = 16384
    c = Cache(rng, dtype, 1, 4, 2, d, [64, 64], cap=cap)
    one = c.tokens(0), c.tokens(1)
    c.tab = np.repeat(c.tab[:, :1], cap, axis=1)
    c.lens = np.full(2, cap * B, np.int32)
    c.upload()
    q = query(rng, 1, 1, 4, d, dtype)
    mass = torch.zeros(c.tab.shape, device="cuda")
    out, lse, status = c.run(q, mass=mass, decay=0.0)
    assert status == 0
    rel = (cap * B / 16 + 16) * 2.0 ** -23  # the additions' bound, as in Cache.check
    for u in range(2):
        K, V, e = one[u]
        want, wl, _, A, S = Q.attend(f64(q)[0, 0, 2 * u:2 * u + 2], K, V, e, np.full(2, B))
        dl = 2.0 ** -18 * S
        assert np.all(np.abs(f64(out)[0, 0, 2 * u:2 * u + 2] - want) <= 2.0 ** -8 * np.abs(want) + (2.0 ** -10 + 2 * rel + 4 * dl[:, None]) * A)
        assert np.all(np.abs(f64(lse)[0, 0, 2 * u:2 * u + 2] - wl - np.log(cap)) <= 3 * dl + 2 * rel)
        assert np.all(np.abs(f64(mass)[u] * cap / 2 - 1) <= 4 * dl.max() + 2 * rel)
