"""What the 4-bit block cache's attention keeps of the bits of its outputs over long caches."""
import numpy as np
import pytest
import torch

from oracle import quant4_oracle as Q
from test_quant4_gpu import Cache
from test_quant_gpu import DT, f64, query

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
