"""Rotary positions and the 4-bit block cache as they are measured: rotating rows, appending tokens, attention.

A 4-bit cache holds `lens` tokens per unit (request b, KV head h): full blocks of 64 tokens as codes n in 0..15 that stand
for (step * n + zero) * scale, and a tail of fewer than 64 tokens in the configuration's type. Keys have a step and a zero
for each channel of a block, values for each token and run of 64 dims, and a block has a power of two (the scale) for its
keys and one for its values. `own` selects between the plain form (torch) and the framework's calls.
"""
import math

import torch

own = False

B = 64  # tokens of a block
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
BASE = 10000.0  # pair i of r / 2 turns by position * BASE^(-2 i / r)


def listed():
    def rotate(name, dtype, batch, hq, hkv, d, tokens, **more):
        return {"name": name, "op": "rotate", "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "tokens": tokens,
                "rot": d, "axes": 1, "interleaved": False, "backward": False, **more}

    def append(name, dtype, batch, hq, hkv, d, tokens, **more):
        return {"name": name, "op": "append", "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "tokens": tokens,
                "ragged": False, "rot": d, "axes": 1, "interleaved": False, **more}

    def attention(name, dtype, batch, hq, hkv, d, ctx, **more):
        return {"name": name, "op": "attention", "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "ctx": ctx,
                "queries": 1, "ragged": False, "mass": False, "rot": 0, "axes": 1, "interleaved": False, **more}

    return [
        # the new token of each of 32 requests, before a decode step: latency counts
        rotate("rotate token 8B", "bf16", 32, 32, 8, 128, 1),
        # the prompts of four requests, before the training-time forward
        rotate("rotate prompt 8B", "bf16", 4, 32, 8, 128, 8192),
        # the gradients of a video's frames: time, height and width, half of the dims, fp32, an odd length
        rotate("rotate video f32 backward", "f32", 3, 8, 2, 64, 1999, rot=32, axes=3, interleaved=True, backward=True),
        # the new token of each of 32 requests
        append("append token 8B", "bf16", 32, 32, 8, 128, 1),
        # the prompts of four requests
        append("append prompt 8B", "bf16", 4, 32, 8, 128, 8192),
        # videos of unequal, odd lengths in fp32
        append("append ragged video f32", "f32", 3, 8, 2, 64, 1999, ragged=True, axes=3),
        # one small fp32 request: launch latency counts
        attention("decode tiny f32", "f32", 1, 4, 1, 64, 2031),
        # a decode step of the 1B-like shape
        attention("decode 1B", "bf16", 8, 16, 8, 64, 16384, rot=64),
        # a decode step of the 3B-like shape, requests of every length, accumulating the blocks' attention weight
        attention("decode 3B ragged mass", "bf16", 16, 24, 8, 128, 32768, ragged=True, mass=True),
        # the offload-heavy 8B-like shape with its whole cache on the GPU
        attention("decode 8B", "bf16", 32, 32, 8, 128, 65536, rot=128),
        # one long request alone
        attention("decode one long", "bf16", 1, 32, 8, 128, 131071, rot=128),
        # eight drafted tokens of four requests verified in one call
        attention("verify 8 tokens", "bf16", 4, 32, 8, 128, 8200, queries=8, rot=128),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attention", "attention", "append", "rotate"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128])
    case = {"op": op, "dtype": rng.choice(["bf16", "bf16", "f32"]), "batch": log(1, 32), "hq": hq, "hkv": hkv, "d": d,
            "rot": rng.choice([d, d, d // 2]), "axes": rng.choice([1, 1, 3]), "interleaved": rng.random() < 0.3}
    if op == "attention":
        queries = rng.choice([1, 1, 1, rng.randint(2, 32)])
        most = min(131072, (1 << 29) // (case["batch"] * hkv * d * max(1, queries * hq // hkv // 8)))
        return {**case, "ctx": log(48, max(64, most)), "queries": queries, "ragged": rng.random() < 0.5, "mass": rng.random() < 0.5,
                "rot": rng.choice([0, case["rot"]])}
    if op == "append":
        most = min(16384, (1 << 25) // (case["batch"] * hkv * d))
        return {**case, "tokens": 1 if rng.random() < 0.3 else log(2, max(4, most)), "ragged": rng.random() < 0.5,
                "rot": rng.choice([0, case["rot"]])}
    most = min(32768, (1 << 27) // (case["batch"] * (hq + hkv) * d))
    return {**case, "tokens": log(1, most), "backward": rng.random() < 0.5}


# ---- what every part shares: lengths and sizes of a case ----------------------------------------------------------
def _lengths(case, most):
    """Tokens of each request: all `most`, or spread over 1..most."""
    n = case["batch"]
    if not case["ragged"]:
        return [most] * n
    return [max(1, most * ((5 * b) % n + 1) // n - 13 * b % 61) for b in range(n)]


def _token_lens(case):
    """Lengths before a single token is appended: every 4th request completes a block."""
    return [4096 + 64 * b + (63 if b % 4 == 0 else 17 * b % 63) for b in range(case["batch"])]


def _unit_bytes(d):
    return -(-(71 * d + 4 * B + 8) // 32) * 32


def _elt(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    d, hq, hkv, elt = case["d"], case["hq"], case["hkv"], _elt(case)
    if case["op"] == "rotate":
        rows = case["batch"] * case["tokens"]
        return {"bytes": float(2 * rows * (hq + hkv) * d * elt + 4 * rows * case["axes"] + 4 * case["tokens"] * case["rot"]),
                "flops": float(3 * rows * (hq + hkv) * case["rot"])}
    block = 71 * d + 4 * B + 8
    if case["op"] == "append":
        new = sum(_lengths(case, case["tokens"]))
        if case["tokens"] == 1:
            full = sum(_token_lens(case)[b] % B == B - 1 for b in range(case["batch"]))
            moved = new * 2 * (2 * d * elt + 4) + full * (B * (2 * d * elt + 4) + block)
        else:
            full = sum(n // B for n in _lengths(case, case["tokens"]))
            moved = new * (2 * d * elt + 4) + full * block + sum(n % B for n in _lengths(case, case["tokens"])) * (2 * d * elt + 4)
        back = full * (block + B * (2 * d * elt + 4))  # the blocks are read back
        return {"bytes": float(hkv * (moved + back) + 4 * new * case["axes"] + 4 * case["tokens"] * case["rot"]),
                "flops": float(hkv * new * (3 * case["rot"] + 8 * d))}
    lens = _lengths(case, case["ctx"])
    rows = case["batch"] * case["queries"] * hq
    nbytes = hkv * sum(n // B * (block + 4) + n % B * (2 * d * elt + 4) for n in lens) + rows * (2 * d * elt + 4)
    if case["mass"]:
        nbytes += hkv * sum(-(-n // B) for n in lens) * 8
    return {"bytes": float(nbytes), "flops": float(4 * d * case["queries"] * hq * sum(lens))}


# ---- the format ----------------------------------------------------------------------------------------------------
def _down16(x):
    """The largest fp16 numbers that are not above x."""
    h = x.half()
    bits = h.view(torch.int16).int()
    bits = torch.where(h.float() > x, torch.where(bits > 0, bits - 1, torch.where(bits == 0, -32767, bits + 1)), bits)
    return bits.short().view(torch.float16).float()


def _up16(x, bits_lost=0):
    """The least fp16 numbers, without their last bits, that are not below x (x >= 0)."""
    h = x.half()
    bits = h.view(torch.int16).int()
    bits = torch.where(h.float() < x, bits + 1, bits)
    low = (1 << bits_lost) - 1
    return ((bits + low) & ~low).short().view(torch.float16).float()


def _scale(x, live):
    """What blocks x [n][64][d] are divided by before they are coded: a power of two that brings the largest magnitude to [4, 8)."""
    a = torch.where(live[..., None], x, 0.0).abs().amax((1, 2))
    power = ((a.view(torch.int32) >> 23) - 2).clamp(min=1) << 23
    return torch.where(a >= 2.0 ** -100, power.view(torch.float32), 0.0)


def _codes(x, live, keys):
    """Codes [n][64][d], steps and zeros (keys: [n][1][d], values: [n][64][d / 64]) and scales [n] of blocks x [n][64][d]."""
    n, _, d = x.shape
    scale = _scale(x, live)
    y = x * torch.where(scale > 0, 1 / scale, 0.0)[:, None, None]
    g = y.view(n, B, d // B, B)
    live = live[..., None]
    if keys:
        lo = torch.where(live, y, math.inf).amin(1, keepdim=True)
        hi = torch.where(live, y, -math.inf).amax(1, keepdim=True)
    else:
        lo, hi = g.amin(-1), g.amax(-1)
    on = (scale > 0)[:, None, None] & (True if keys else live)
    zero = torch.where(on, _down16(torch.where(on, lo, 0.0)), 0.0)
    fifteenth = torch.tensor(1 / 15, device=x.device)
    step = torch.where(on, _up16((torch.where(on, hi, 0.0) - zero) * fifteenth, 8 if keys else 0), 0.0)
    inv = torch.where(step > 0, 1 / step, 0.0)
    z, r = (zero, inv) if keys else (t[..., None].expand(g.shape).reshape(y.shape) for t in (zero, inv))
    codes = ((y - z).double() * r.double()).round()  # in 64 bits: borders
    return torch.where(on.any(-1, keepdim=True) & live, codes, 0.0).to(torch.uint8), step, zero, scale


def _values(codes, step, zero, scale, keys):
    """The values that codes stand for, in fp32."""
    x = codes.float()
    if keys:
        return x.mul_(step).add_(zero).mul_(scale[..., None, None])
    g = x.view(*x.shape[:-1], x.shape[-1] // B, B)
    return g.mul_(step[..., None]).add_(zero[..., None]).mul_(scale[..., None, None, None]).view(x.shape)


def _image(kc, ks, kz, kscale, vc, vs, vz, vscale, e):
    """Block units: the layout that the header documents."""
    n, d = kc.shape[0], kc.shape[-1]
    m = d // 16
    img = torch.zeros(n, _unit_bytes(d), dtype=torch.uint8, device=kc.device)

    def words(codes):  # [n][m][32 lanes][4 slices][8]: the codes of a word, lowest bits first
        c = codes.reshape(n, m, 32, 4, 4, 2)
        return (c[..., 0] | c[..., 1] << 4).reshape(n, -1)

    # keys: tokens (w, t2, half, t0), dims (m, c, i1, i0) -> m, lane (t2, t0, c), w, nibble (i0, i1, half)
    img[:, : 32 * d] = words(kc.view(n, 4, 4, 2, 2, m, 4, 2, 2).permute(0, 5, 2, 4, 6, 1, 8, 7, 3).contiguous())
    # values: tokens (w, c, i1, i0), dims (m, half, g) -> m, lane (g, c), w, nibble (i0, i1, half)
    img[:, 32 * d : 64 * d] = words(vc.view(n, 4, 4, 2, 2, m, 2, 8).permute(0, 5, 7, 2, 1, 4, 3, 6).contiguous())
    ordered = lambda x: x.reshape(n, -1, 4, 4).transpose(1, 2).reshape(n, -1)  # noqa: E731
    img[:, 64 * d : 65 * d] = ordered(ks.view(n, d)).half().view(torch.int16).int().bitwise_right_shift(8).to(torch.uint8)
    img[:, 65 * d : 67 * d] = ordered(kz.view(n, d)).half().contiguous().view(torch.uint8)
    for at, x in ((67 * d, vs), (69 * d, vz)):
        x = torch.cat([ordered(x[..., i]) for i in range(d // B)], 1)
        img[:, at : at + 2 * d] = x.half().contiguous().view(torch.uint8)
    img[:, 71 * d : 71 * d + 4 * B] = e.contiguous().view(torch.uint8)
    img[:, 71 * d + 4 * B : 71 * d + 4 * B + 8] = torch.stack([kscale, vscale], 1).contiguous().view(torch.uint8)
    return img


# ---- inputs --------------------------------------------------------------------------------------------------------
def _tail_bytes(d, elt):
    return -(-(2 * B * d * elt + 4 * B) // 256) * 256


def _tail_parts(tail, d, dtype):
    """Views of tail units: keys [U][d / c][64][c] (c elements are 16 bytes), values [U][64][d], logits [U][64]."""
    elt = torch.empty(0, dtype=dtype).element_size()
    kb = B * d * elt
    u = tail.shape[0]
    return (tail[:, :kb].view(dtype).view(u, d * elt // 16, B, 16 // elt), tail[:, kb : 2 * kb].view(dtype).view(u, B, d),
            tail[:, 2 * kb : 2 * kb + 4 * B].view(torch.float32))


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _logits(g, *shape):
    """Eviction logits, N(0, 1); one token in a hundred is masked."""
    e = _normal(g, *shape)
    return torch.where(torch.rand(*shape, generator=g, device="cuda") < 0.01, -math.inf, e)


def _keys(g, *shape):
    """Keys: channels with means of their own, one in sixteen of them large."""
    d = shape[-1]
    mean = _normal(g, d) * torch.where(torch.arange(d, device="cuda") % 16 == 5, 4.0, 0.5)
    return _normal(g, *shape).add_(mean)


def _per_unit(case, per_request):
    return torch.tensor(per_request, dtype=torch.int32, device="cuda").repeat_interleave(case["hkv"]).contiguous()


def _axes(case):
    """Axis of each pair: a quarter of the pairs time, the rest height and width; or one axis."""
    pairs = case["rot"] // 2
    t, h = pairs // 4, (pairs - pairs // 4) // 2
    return [0] * pairs if case["axes"] == 1 else [0] * t + [1] * h + [2] * (pairs - t - h)


def _positions(case, first):
    """Positions [axes][batch][n] of tokens from `first` [batch] on: their number, or frames of 18 x 30 patches."""
    p = torch.tensor(first, device="cuda")[:, None] + torch.arange(case.get("tokens", case.get("queries")), device="cuda")
    p = p[None] if case["axes"] == 1 else torch.stack([p // 540, p // 30 % 18, p % 30])
    return p.to(torch.int32).contiguous()


def _rotation(case, first, s):
    """Into the state: positions, the axes of the pairs, and the table [positions][rot / 2][2] of cosines and sines."""
    if not case["rot"]:
        return
    s["pos"] = _positions(case, first)
    s["axis"] = _axes(case)
    pairs = case["rot"] // 2
    turn = BASE ** (-torch.arange(pairs, dtype=torch.float64, device="cuda") / pairs)
    a = torch.arange(int(s["pos"].max()) + 1, dtype=torch.float64, device="cuda")[:, None] * turn
    s["table"] = torch.stack([a.cos(), a.sin()], -1).float()
    s["axis_index"] = torch.tensor(s["axis"], device="cuda")


def _config(case):
    import trainable_sparse_attention_decode_gb300 as nosa
    return nosa.nosa_config(case["batch"], case["hq"], case["hkv"], case["d"], case["dtype"], 1, 0, 64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    U = case["batch"] * case["hkv"]
    d, dtype = case["d"], TYPES[case["dtype"]]
    b, hkv = case["batch"], case["hkv"]
    if case["op"] == "rotate":
        n = case["tokens"]
        # single tokens stand at lengths of their own, prompts start at 0
        _rotation(case, _token_lens(case) if n == 1 else [0] * b, s)
        s["q"] = _normal(g, b, n, case["hq"], d).to(dtype)
        s["k"] = _keys(g, b, n, hkv, d).to(dtype)
        s["q_out"], s["k_out"] = torch.empty_like(s["q"]), torch.empty_like(s["k"])
        return s
    s["tail"] = torch.zeros(U, _tail_bytes(d, _elt(case)), dtype=torch.uint8, device="cuda")
    tk, tv, te = _tail_parts(s["tail"], d, dtype)
    if case["op"] == "append":
        n = case["tokens"]
        old = _token_lens(case) if n == 1 else [0] * b
        s["lens"] = _per_unit(case, old)
        _rotation(case, old, s)
        if n == 1:  # the tails hold tokens already
            tk.copy_(_normal(g, *tk.shape))
            tv.copy_(_normal(g, *tv.shape))
            te.copy_(_logits(g, *te.shape))
        # one unit for each block that the call may complete; the entries before them are not this call's
        count = _lengths(case, n)
        new = max(1, n // B)
        first = max(old) // B
        s["tab"] = torch.full((U, first + new + 1), -1, dtype=torch.int32, device="cuda")
        at = (s["lens"] // B)[:, None].long() + torch.arange(new, device="cuda")
        perm = torch.randperm(U * new, generator=g, device="cuda").to(torch.int32).view(U, new)
        s["tab"].scatter_(1, at, perm)
        done = _per_unit(case, [(o % B + m) // B for o, m in zip(old, count)])
        s["ids"] = perm[torch.arange(new, device="cuda") < done[:, None]]  # the units that the call fills
        s["units"] = torch.zeros(U * new, _unit_bytes(d), dtype=torch.uint8, device="cuda")
        s["k"] = _keys(g, b, n, hkv, d).to(dtype)
        s["v"] = _normal(g, b, n, hkv, d).to(dtype)
        s["e"] = _logits(g, b, n, hkv)
        s["n_new"] = torch.tensor(count, dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["lens_out"] = torch.empty_like(s["lens"])
        s["k_back"] = torch.empty(s["ids"].shape[0], B, d, dtype=dtype, device="cuda")
        s["v_back"], s["e_back"] = torch.empty_like(s["k_back"]), torch.empty(s["ids"].shape[0], B, device="cuda")
        return s
    lens = _lengths(case, case["ctx"])
    s["lens"] = _per_unit(case, lens)
    _rotation(case, [max(0, n - case["queries"]) for n in lens], s)
    tk.copy_(_normal(g, *tk.shape))
    tv.copy_(_normal(g, *tv.shape))
    te.copy_(_logits(g, *te.shape))
    blocks = [n // B for n in lens for _ in range(hkv)]
    cap = max(-(-max(lens) // B), 1)
    total = sum(blocks)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(blocks, device="cuda")
    at = torch.arange(cap, device="cuda")[None] + (count.cumsum(0) - count)[:, None]
    s["tab"] = torch.where(torch.arange(cap, device="cuda")[None] < count[:, None], perm[at.clamp(max=max(total - 1, 0))] if total else -1, -1)
    s["tab"] = s["tab"].to(torch.int32).contiguous()
    s["kc"] = torch.empty(total, B, d, dtype=torch.uint8, device="cuda")
    s["vc"] = torch.empty(total, B, d, dtype=torch.uint8, device="cuda")
    s["kp"] = torch.empty(2, total, 1, d, device="cuda")       # steps and zeros of the keys' channels
    s["vp"] = torch.empty(2, total, B, d // B, device="cuda")  # ... and of the values' tokens
    s["scales"] = torch.empty(2, total, device="cuda")
    s["e"] = _logits(g, total, B)
    s["units"] = torch.empty(total, _unit_bytes(d), dtype=torch.uint8, device="cuda")
    for i in range(0, total, 1 << 15):  # a part at a time, so that the fp32 values need little room
        p = slice(i, min(total, i + (1 << 15)))
        m = p.stop - p.start
        live = s["e"][p] > -math.inf
        k = _codes(_keys(g, m, B, d), live, True)
        v = _codes(_normal(g, m, B, d), live, False)
        s["units"][p] = _image(*k, *v, s["e"][p])
        s["kc"][p], s["kp"][0][p], s["kp"][1][p], s["scales"][0][p] = k
        s["vc"][p], s["vp"][0][p], s["vp"][1][p], s["scales"][1][p] = v
    s["q"] = _normal(g, b, case["queries"], case["hq"], d).to(dtype)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:3], device="cuda")
    s["mass"] = torch.rand(U, cap, generator=g, device="cuda") if case["mass"] else None
    return s


def _plan(s, make):
    """The configuration, rotation and workspace that a program keeps: made by the first call on a state."""
    if "plan" not in s:
        s["plan"] = make()
    return s["plan"]


def _rope(s):
    import trainable_sparse_attention_decode_gb300 as nosa
    return nosa.nosa_rope(s["table"], axes=s["axis"], interleaved=s["case"]["interleaved"]) if s["case"]["rot"] else None


DECAY = 0.96875


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    return {"rotate": _rotate, "append": _append, "attention": _attention}[s["case"]["op"]](s)


def _turn(s, x, backward=False):
    """Rows x [batch][n][heads][d] turned by their positions, in fp32, rounded to their type."""
    case = s["case"]
    r = case["rot"]
    if not r:
        return x
    cs = s["table"][s["pos"].long()[s["axis_index"]], torch.arange(r // 2, device="cuda")[:, None, None]]  # [r / 2][batch][n][2]
    c, z = cs.permute(1, 2, 0, 3)[:, :, None].unbind(-1)
    if backward:
        z = -z
    y = x.float()
    a, b = (y[..., 0:r:2], y[..., 1:r:2]) if case["interleaved"] else (y[..., : r // 2], y[..., r // 2 : r])
    a, b = a * c - b * z, b * c + a * z
    turned = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([turned, y[..., r:]], -1).to(x.dtype)


def _rotate(s):
    if own:
        import trainable_sparse_attention_decode_gb300 as nosa
        cfg, rope = _plan(s, lambda: (_config(s["case"]), _rope(s)))
        nosa.nosa_rotate(cfg, rope, s["pos"], s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"], backward=s["case"]["backward"])
    else:
        s["q_out"].copy_(_turn(s, s["q"], s["case"]["backward"]))
        s["k_out"].copy_(_turn(s, s["k"], s["case"]["backward"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def _append(s):
    case = s["case"]
    d, dtype = case["d"], TYPES[case["dtype"]]
    tk, tv, te = _tail_parts(s["tail"], d, dtype)
    result = {"k": s["k_back"], "v": s["v_back"], "e": s["e_back"], "tail_k": tk, "tail_v": tv, "tail_e": te, "lens": s["lens_out"]}
    if own:
        import trainable_sparse_attention_decode_gb300 as nosa
        cfg, rope = _plan(s, lambda: (_config(case), _rope(s)))
        nosa.nosa_quant4_append(cfg, s["k"], s["v"], s["e"], s["units"], s["tab"], s["tail"], s["lens"], s["lens_out"],
                                n_new=s["n_new"], rope=rope, positions=s.get("pos"))
        nosa.nosa_quant4_read(cfg, s["units"], s["k_back"], s["v_back"], s["e_back"], ids=s["ids"])
        return result
    b, n, hkv = case["batch"], case["tokens"], case["hkv"]
    U = b * hkv
    lens = s["lens"].long()
    new = s["n_new"].long().repeat_interleave(hkv) if s["n_new"] is not None else torch.full_like(lens, n)
    rows = lambda x: x.transpose(1, 2).reshape(U, n, -1)  # noqa: E731
    k, v, e = rows(_turn(s, s["k"])), rows(s["v"]), rows(s["e"][..., None])[..., 0]
    # the tails with the new tokens behind them: [U][64 + n]
    blocks = (B + n) // B
    at = torch.arange((blocks + 1) * B, device="cuda") - (lens % B)[:, None]
    mine = (at >= 0) & (at < new[:, None])
    pick = at.clamp(0, n - 1)

    def behind(old, x):
        x = x.gather(1, pick.view(pick.shape + (1,) * (x.ndim - 2)).expand(pick.shape + x.shape[2:]))
        was = torch.zeros_like(x)
        was[:, :B] = old
        return torch.where(mine.view(mine.shape + (1,) * (x.ndim - 2)), x, was)

    k = behind(tk.transpose(1, 2).reshape(U, B, d), k).view(U, blocks + 1, B, d)
    v = behind(tv, v).view(U, blocks + 1, B, d)
    e = behind(te, e).view(U, blocks + 1, B)
    done = ((lens % B + new) // B)[:, None]  # blocks completed
    j = torch.arange(blocks, device="cuda")
    to = s["tab"].gather(1, ((lens // B)[:, None] + j).clamp(max=s["tab"].shape[1] - 1)).long()
    full = (j < done).view(-1)
    place = torch.zeros(s["units"].shape[0], dtype=torch.long, device="cuda")
    place[to.view(-1)[full]] = torch.arange(U * blocks, device="cuda")[full]
    read = place[s["ids"].long()]  # where the blocks that are read back stand
    eb = e[:, :blocks].reshape(-1, B)[read]
    live = eb > -math.inf
    for x, out, keys in ((k, s["k_back"], True), (v, s["v_back"], False)):
        y = _values(*_codes(x[:, :blocks].reshape(-1, B, d)[read].float(), live, keys), keys)
        out.copy_(torch.where(live[..., None], y, 0.0))
    s["e_back"].copy_(eb)
    # what is left becomes the tails; rows behind them stay
    left = (lens % B + new - done[:, 0] * B)[:, None]
    take = lambda x: x.gather(1, done.view(U, 1, *[1] * (x.ndim - 2)).expand(U, 1, *x.shape[2:]))[:, 0]  # noqa: E731
    keep = torch.arange(B, device="cuda") < left
    tk.copy_(torch.where(keep[:, None, :, None], take(k).view(U, B, tk.shape[1], tk.shape[3]).transpose(1, 2), tk))
    tv.copy_(torch.where(keep[..., None], take(v), tv))
    te.copy_(torch.where(keep, take(e), te))
    s["lens_out"].copy_(s["lens"] + new.to(torch.int32))
    return result


def _attention(s):
    case = s["case"]
    result = {"out": s["out"], "lse": s["lse"]}
    if s["mass"] is not None:
        result["mass"] = s["mass"]
    if own:
        import trainable_sparse_attention_decode_gb300 as nosa
        cfg, rope, ws = _plan(s, lambda: (c := _config(case), _rope(s), torch.empty(
            nosa.nosa_quant4_attention_workspace_bytes(c, s["tab"].shape[1], case["queries"], case["mass"]),
            dtype=torch.uint8, device="cuda")))
        nosa.nosa_quant4_attention(cfg, s["units"], s["tab"], s["tail"], s["lens"], s["q"], s["out"], lse=s["lse"],
                                   mass=s["mass"], decay=DECAY, rope=rope, positions=s.get("pos"), workspace=ws)
        return result
    b, T, hq, hkv, d = case["batch"], case["queries"], case["hq"], case["hkv"], case["d"]
    U, G, R = b * hkv, hq // hkv, T * hq // hkv
    cap = s["tab"].shape[1]
    q = _turn(s, s["q"]).float().view(b, T, hkv, G, d).transpose(1, 2).reshape(U, R, d) / math.sqrt(d)
    # the positions of the full blocks, and of the tails
    lens = s["lens"].long()
    full = lens // B * B
    sees = (lens[:, None] - T + 1 + torch.arange(T, device="cuda")).repeat_interleave(G, 1)[..., None]  # [U][R][1]
    pos = torch.arange(cap * B, device="cuda")
    tpos = full[:, None, None] + torch.arange(B, device="cuda")
    tk, tv, te = _tail_parts(s["tail"], d, TYPES[case["dtype"]])
    tk = tk.transpose(1, 2).reshape(U, B, d).float()
    tlive = tpos < torch.minimum(sees, lens[:, None, None])
    logits = [torch.where(tlive, q @ tk.transpose(1, 2) + te[:, None], -math.inf)]
    if s["kc"].shape[0]:
        tab = s["tab"].clamp(min=0).long()
        k = _values(s["kc"][tab], s["kp"][0][tab], s["kp"][1][tab], s["scales"][0][tab], True)
        l = (q @ k.view(U, cap * B, d).transpose(1, 2)).add_(s["e"][tab].view(U, 1, cap * B))
        del k
        logits.append(torch.where(pos < torch.minimum(sees, full[:, None, None]), l, -math.inf))
        del l
    m = torch.stack([x.amax(-1) for x in logits]).amax(0)
    m = torch.where(m == -math.inf, 0.0, m)[..., None]
    w = [torch.exp(x - m) for x in logits]
    del logits
    z = sum(x.sum(-1, keepdim=True) for x in w)
    w = [x.div_(torch.where(z > 0, z, 1.0)) for x in w]
    o = w[0] @ torch.where(tlive.any(1)[..., None], tv.float(), 0.0)
    mass = torch.zeros(U, cap + 1, device="cuda")
    if len(w) > 1:
        mass[:, :cap] = w[1].view(U, R, cap, B).sum((1, 3))
        v = _values(s["vc"][tab], s["vp"][0][tab], s["vp"][1][tab], s["scales"][1][tab], False)
        o = o + w[1] @ v.view(U, cap * B, d)
    mass.scatter_add_(1, (lens // B)[:, None], w[0].sum((1, 2))[:, None])
    heads = lambda x: x.view(b, hkv, T, G, -1).transpose(1, 2).reshape(b, T, hq, -1)  # noqa: E731
    s["out"].copy_(heads(o))
    s["lse"].copy_(heads(m + torch.log(z))[..., 0])
    if s["mass"] is not None:
        s["mass"].mul_(DECAY).add_(mass[:, :cap])
    return result


# ---- the definition in 64 bits ------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rotate": _exact_rotate, "append": _exact_append, "attention": _exact_attention}[case["op"]](case, s)


def _exact_turn(case, s, x, sign=1.0):
    """Every pair as a complex number times that of its angle."""
    y = x.to(torch.float64).clone()
    for i, axis in enumerate(s.get("axis", [])):
        at = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + case["rot"] // 2)
        t = s["table"][s["pos"][axis].long(), i].to(torch.float64)
        z = torch.complex(y[..., at[0]], y[..., at[1]]) * torch.complex(t[..., 0], sign * t[..., 1])[:, :, None]
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
    return y


def _exact_rotate(case, s):
    sign = -1.0 if case["backward"] else 1.0
    return {"q": _exact_turn(case, s, s["q"], sign), "k": _exact_turn(case, s, s["k"], sign)}


def _exact_groups(x):
    """Groups x [n][64] of numbers below 8 in size as 4-bit codes, zeros and steps apart: (zero, room above it)."""
    lo, hi = x.amin(1), x.amax(1)
    unit = torch.exp2(torch.floor(torch.log2(lo.abs().clamp(min=2.0 ** -14))) - 10)  # spacing of fp16 numbers there
    zero = torch.floor(lo / unit) * unit
    return zero, ((hi - zero).float() * torch.tensor(1 / 15, device=x.device)).to(torch.float64)


def _exact_step(room, bits):
    """The least numbers of so many significant bits, of fp16's range, that are not below `room`."""
    unit = torch.exp2(torch.floor(torch.log2(room.clamp(min=2.0 ** -14))) - (bits - 1))
    return torch.ceil(room / unit) * unit


def _exact_coded(x, keys, live):
    """What a block x [64][d] reads back as, from the format's definition; None-valued tokens read 0."""
    f64 = torch.float64
    top = x[live].abs().max() if live.any() else torch.zeros((), dtype=f64, device=x.device)
    if top < 2.0 ** -100:
        return torch.zeros_like(x)
    scale = torch.exp2(torch.floor(torch.log2(top)) - 2)
    y = torch.where(live[:, None], x / scale, 0.0)
    d = y.shape[1]
    if keys:
        groups = y[live].T
    else:
        groups = y[live].reshape(-1, B)
    zero, room = _exact_groups(groups)
    step = _exact_step(room, 3 if keys else 11)
    inv = torch.where(step > 0, (1 / step).float().to(f64), 0.0)
    n = torch.round((groups - zero[:, None]).float().to(f64) * inv[:, None])
    back = (n * step[:, None] + zero[:, None]) * scale
    out = torch.zeros_like(x)
    out[live] = back.T if keys else back.reshape(-1, d)
    return out


def _exact_append(case, s):
    d, hkv, dtype = case["d"], case["hkv"], TYPES[case["dtype"]]
    f64 = torch.float64
    U = case["batch"] * hkv
    if s["ids"].shape[0] > 8192:
        return None
    keys = _exact_turn(case, s, s["k"])
    rounded = keys.to(dtype)
    tk, tv, te = [x.to(f64) for x in _tail_parts(s["tail"], d, dtype)]
    lens = s["lens"].tolist()
    new = s["n_new"].tolist() if s["n_new"] is not None else [case["tokens"]] * case["batch"]
    units = s["units"].shape[0]
    back = torch.zeros(2, units, B, d, dtype=f64, device="cuda")
    logits = torch.zeros(units, B, dtype=f64, device="cuda")
    after = []
    for u in range(U):
        b, h = u // hkv, u % hkv
        n0, n1 = lens[u], lens[u] + new[b]
        after.append(n1)
        old = n0 % B
        unrounded = torch.cat([tk[u].permute(1, 0, 2).reshape(B, d)[:old], keys[b, : new[b], h]])
        k = torch.cat([tk[u].permute(1, 0, 2).reshape(B, d)[:old], rounded[b, : new[b], h].to(f64)])
        v = torch.cat([tv[u, :old], s["v"][b, : new[b], h].to(f64)])
        e = torch.cat([te[u, :old], s["e"][b, : new[b], h].to(f64)])
        done = k.shape[0] // B
        for i, to in enumerate(s["tab"][u, n0 // B : n0 // B + done].tolist()):
            p = slice(i * B, i * B + B)
            live = e[p] > -math.inf
            logits[to] = e[p]
            back[0, to], back[1, to] = _exact_coded(k[p], True, live), _exact_coded(v[p], False, live)
        left = k.shape[0] - done * B
        first = old if not done else 0  # a tail that goes on keeps its rows
        if left > first:
            rows = slice(done * B + first, done * B + left)
            tk[u][:, first:left] = unrounded[rows].view(left - first, tk.shape[1], tk.shape[3]).transpose(0, 1)
            tv[u][first:left] = v[rows]
            te[u][first:left] = e[rows]
    ids = s["ids"].long()
    # (a rotated fp32 key is a rounding off, which decides a code where it lies that near to a border)
    k = None if dtype == torch.float32 and case["rot"] else back[0][ids]
    return {"k": k, "v": back[1][ids], "e": logits[ids], "tail_k": tk, "tail_v": tv, "tail_e": te,
            "lens": torch.tensor(after, dtype=torch.int32, device="cuda")}


def _exact_attention(case, s):
    T, hq, hkv, d = case["queries"], case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    f64 = torch.float64
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=f64, device="cuda")
    mass = None if s["mass"] is None else s["mass"].to(f64) * DECAY
    tk, tv, te = _tail_parts(s["tail"], d, TYPES[case["dtype"]])
    q = _exact_turn(case, s, s["q"]).to(s["q"].dtype).to(f64)  # a rotated query is rounded to its type
    lens = s["lens"].tolist()
    for u, n in enumerate(lens):
        b, h = u // hkv, u % hkv
        nb, nt = n // B, n % B
        ids = s["tab"][u, :nb].long()
        sk, sv = s["scales"][:, ids].to(f64)
        keys = ((s["kc"][ids].to(f64) * s["kp"][0, ids].to(f64) + s["kp"][1, ids].to(f64)) * sk.view(-1, 1, 1)).view(nb * B, d)
        vals = s["vc"][ids].to(f64).view(nb, B, d // B, B) * s["vp"][0, ids].to(f64)[..., None]
        vals = ((vals + s["vp"][1, ids].to(f64)[..., None]) * sv.view(-1, 1, 1, 1)).view(nb * B, d)
        keys = torch.cat([keys, tk[u].to(f64).permute(1, 0, 2).reshape(B, d)[:nt]])
        vals = torch.cat([vals, tv[u, :nt].to(f64)])
        bias = torch.cat([s["e"][ids].view(-1), te[u, :nt]]).to(f64)
        qs = q[b, :, h * G : (h + 1) * G].reshape(T * G, d)
        logit = torch.matmul(qs, keys.T) * d ** -0.5 + bias
        last = n - T + torch.arange(T * G, device="cuda") // G
        logit.masked_fill_(torch.arange(n, device="cuda")[None] > last[:, None], -math.inf)
        total = torch.logsumexp(logit, 1, keepdim=True)
        p = torch.where(total > -math.inf, torch.exp(logit - total), 0.0)
        out[b, :, h * G : (h + 1) * G] = torch.matmul(p, vals).view(T, G, d)
        lse[b, :, h * G : (h + 1) * G] = total.view(T, G)
        if mass is not None:
            per = p.sum(0)
            mass[u, :nb] += per[: nb * B].view(nb, B).sum(1)
            if nt:
                mass[u, nb] += per[nb * B :].sum()
    res = {"out": out, "lse": lse}
    if mass is not None:
        res["mass"] = mass
    return res
