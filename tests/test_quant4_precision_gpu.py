"""What the 4-bit block cache's attention keeps of the bits of its logits and outputs: long caches, lopsided
queries, large values."""
import numpy as np
import pytest
import torch

from oracle import quant4_oracle as Q
from test_quant4_gpu import Cache
from test_quant_gpu import B, DT, f64, query

pytestmark = pytest.mark.gpu


def own_rounding(want):
    """The errors that rounding fp64 outputs to bf16 makes."""
    return f64(torch.as_tensor(want).to(DT["bf16"])) - want


@pytest.mark.parametrize("d,hkv,T,n", [(64, 2, 1, 65536), (128, 1, 1, 65536), (64, 2, 1, 131071), (128, 1, 4, 131071)])
def test_bf16_outputs_of_long_caches(d, hkv, T, n):
    """bf16 outputs over 65536 tokens and more are off by their own rounding and little else.

    The values are independent and of both signs, so a row's sum has the size sqrt(sum w_j^2) of a value's. Its terms
    are off by two independent roundings to 11 bits, each 0.42 * 2^-11 in the mean square of what it rounds (half a
    step is 2^-11 of a number at most): the weight's, of w_j v_j, and that of its product with the step, of w_j step_j
    n_jx, which is 2.6 times w_j v_jx for a normal sample's 16 levels. Together 1.17 * 2^-11 of the output in the
    norm. The output's own rounding is taken from the fp64 outputs rounded to bf16: sums of N >= 1024 squares of
    rounding errors differ by less than 15 % (4 standard deviations)."""
    rng = np.random.default_rng(n + d + T)
    c = Cache(rng, "bf16", 1, 8 * hkv, hkv, d, [n] * hkv, masked=0.0).upload()
    q = query(rng, 1, T, 8 * hkv, d, "bf16")
    out, lse, status = c.run(q)
    assert status == 0
    want = np.empty(q.shape)
    for u in range(hkv):
        K, V, e, Ks, Vs = c.tokens(u)
        rows = f64(q)[0, :, 8 * u:8 * u + 8].reshape(8 * T, d)
        want[0, :, 8 * u:8 * u + 8] = Q.attend(rows, K, V, e, np.repeat(n - T + 1 + np.arange(T), 8), Ks, Vs)[0].reshape(T, 8, d)
    err, own = f64(out) - want, own_rounding(want)
    assert (err ** 2).sum() <= 1.15 * (own ** 2).sum() + (1.25 * 2.0 ** -11) ** 2 * (want ** 2).sum()


@pytest.mark.parametrize("d", [64, 128])
def test_bf16_outputs_are_not_off_to_one_side(d):
    """Outputs over 131072 values of both signs are not smaller or larger than they are on the whole.

    A product of a weight (times its step) and a code is cut off, towards zero, 2^-25 below the largest of the sixteen
    tokens' that are added at once, where a code's exponent is written as 2^6 at most (raised by 2^4; without that 2^10 in
    the dims x with x % 16 < 8): half of 2^-19 of the largest weight times step of the sixteen, for each of them, in the
    mean. The output's own rounding has mean 0 but for 4 standard deviations, its size over the root of the number
    of outputs."""
    n, T = 131072, 8
    rng = np.random.default_rng(d)
    c = Cache(rng, "bf16", 1, 8, 1, d, [n], masked=0.0).upload()
    q = query(rng, 1, T, 8, d, "bf16")
    out, lse, status = c.run(q)
    assert status == 0
    K, V, e, Ks, Vs = c.tokens(0)
    want, _, w, _, _ = Q.attend(f64(q)[0].reshape(-1, d), K, V, e, np.repeat(n - T + 1 + np.arange(T), 8), Ks, Vs)
    _, (_, step, _), scales, _ = Q.parts(c.images[c.tab[0]], d)
    step = (step * scales[:, 1, None, None]).reshape(n, d).max(1)
    lost = 16 * 2.0 ** -20 * (w * step).reshape(len(w), -1, 16).max(2).sum(1).mean()
    err, own = f64(out)[0].reshape(-1, d) - want, own_rounding(want)
    for half in (0, 1):
        dims = np.arange(d) % 16 // 8 == half
        noise = 4 * np.sqrt((own[:, dims] ** 2).mean() / own[:, dims].size)
        assert abs(err[:, dims].mean()) <= lost + noise, half


def one_block(d, codes, steps, zeros, token):
    """The image of a block of keys `codes` [64][d] with these steps and zeros [d], values 0, in which one token counts."""
    img = np.zeros((1, Q.unit_bytes(d)), np.uint8)
    (kb, ks), _ = Q.code_places(d)
    for half in (0, 4):
        own = ks == half
        img[0, kb[own]] |= (codes[own] << half).astype(np.uint8)
    p = Q.places(d)
    img[0, p[0]] = steps.astype(np.float16).view(np.uint16) >> 8
    bits = zeros.astype(np.float16).view(np.uint16)
    img[0, p[1]], img[0, p[1] + 1] = bits & 255, bits >> 8
    e = np.full(B, -np.inf, np.float32)
    e[token] = 0
    img[0, 71 * d:71 * d + 4 * B + 8] = np.concatenate([e, np.ones(2, np.float32)]).view(np.uint8)
    return img


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["one channel", "one channel, mostly zeros", "every 16th channel", "zeros of all sizes"])
def test_single_logits_of_lopsided_queries(dtype, d, kind):
    """A logit is off by at most 2^-18 of the sum over dims of |q| (15 step + |zero|), also of a token whose own sum is far
    smaller: channels whose query element is up to 2^24 times the others', and whose codes and zeros may be 0.

    A product of sixteen is cut off 2^-25 below the largest, whose operand's exponent is written as 2^6 for a code
    at most: with M the largest |q| step of the sixteen dims, 17 terms of 2^-19 M, and a seventeenth of that for the
    neighbour's code, for d / 16 sums: 2^-14.8 of the sum of the M, of which the bound's sum is at least 15 times: 2^-18.7.
    The zeros' products add 17 * 2^-25, in fp32 the partial sums of three terms 3 d / 16 * 2^-24 (and the codes, as
    normal numbers, less), and the logit its last three roundings."""
    U = 64
    for boost in range(0, 25, 3):
        rng = np.random.default_rng(boost)
        codes = np.where(rng.random((B, d)) < 0.5, 15, rng.integers(0, 16, size=(B, d)))
        steps, zeros = np.full(d, 0.5), np.zeros(d)
        big = np.arange(d) == 3
        if kind == "one channel":
            codes[:, 3] = np.where(np.arange(B) == 0, 15, rng.integers(1, 16, size=B))
        elif kind == "one channel, mostly zeros":
            codes[:, 3] = np.where(np.arange(B) == 0, 15, rng.integers(0, 2, size=B) * (np.arange(B) % 2))
        elif kind == "every 16th channel":
            codes[0::3], codes[1::3] = 15, 0
            big = np.arange(d) % 16 == 0
        else:
            zeros = f64(torch.as_tensor(rng.normal(size=d)).half())
        c = Cache(rng, dtype, U, 8, 1, d, [B] * U, masked=0.0)
        c.images = np.concatenate([one_block(d, codes, steps, zeros, t) for t in range(U)])
        c.tab = np.arange(U, dtype=np.int32)[:, None].copy()
        c.upload()
        q = np.abs(rng.normal(size=(1, 1, 8, d))) + 0.3
        q[..., 4:] *= np.where(rng.random(d - 4) < 0.2, -1, 1)
        q = torch.as_tensor(np.repeat(np.where(big, q * 2.0 ** boost, q), U, 0)).to(DT[dtype]).cuda()
        out, lse, status = c.run(q)
        assert status == 0
        rows = f64(q)[0, 0]
        want = rows @ (codes * steps + zeros).T / np.sqrt(d)
        most = np.abs(rows) @ (15 * steps + np.abs(zeros)) / np.sqrt(d)
        assert np.all(np.abs(f64(lse)[:, 0].T - want) <= 2.0 ** -18 * most[:, None] + 2.0 ** -22 * np.abs(want)), boost


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f32", 64), ("f32", 128), ("bf16", 64)])
@pytest.mark.parametrize("n,T", [(4096 - 10, 1), (64, 1), (64, 64), (4, 2)])
def test_values_as_large_as_the_tokens_allow(dtype, d, n, T):
    """Values whose number in the unit times their size stays below 2^126 do not leave fp32's range in the sums, where a
    row sees all of the tokens, one of them, or only a tail."""
    rng = np.random.default_rng(n)
    c = Cache(rng, dtype, 1, 4, 1, d, [n], masked=0.0)
    size = 2.0 ** (125 - np.ceil(np.log2(n)))
    v = size * rng.uniform(1.0, 1.98, size=(len(c.images), B, d))
    c.images = Q.encode(rng.normal(size=v.shape), v, np.zeros((len(v), B)))
    c.tv = f64(torch.as_tensor(size * rng.uniform(1.0, 1.98, size=c.tv.shape)).to(DT[dtype]))
    c.te[:] = 0
    c.upload()
    q = torch.zeros(1, T, 4, d, dtype=DT[dtype], device="cuda")
    out, lse, status = c.run(q)
    assert status == 0
    c.check(q, out, lse)
