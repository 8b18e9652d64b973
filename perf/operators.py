"""The operators of the 8-bit block cache as they are measured: appending tokens, attention over the cache, eviction.

Each case is one call of one operator on a cache whose units (request b, KV head h) hold `lens` tokens: full blocks of
64 tokens in 8 bits with one scale for the keys and one for the values of each block and head, and a tail of fewer than
64 tokens in the configuration's type. `own` selects between the plain form (torch) and the framework's calls.
"""
import math

import torch

own = False

B = 64  # tokens of a block
E4M3 = torch.float8_e4m3fn
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    def attention(name, dtype, batch, hq, hkv, d, ctx, **more):
        return {"name": name, "op": "attention", "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "ctx": ctx,
                "queries": 1, "ragged": False, "mass": False, **more}

    def append(name, dtype, batch, hq, hkv, d, tokens, **more):
        return {"name": name, "op": "append", "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d,
                "tokens": tokens, "ragged": False, **more}

    return [
        # one small fp32 request: launch latency counts
        attention("decode tiny f32", "f32", 1, 4, 1, 64, 2031),
        # a decode step of the 1B-like shape
        attention("decode 1B", "bf16", 8, 16, 8, 64, 16384),
        # a decode step of the 3B-like shape, requests of every length, accumulating the blocks' attention weight
        attention("decode 3B ragged mass", "bf16", 16, 24, 8, 128, 32768, ragged=True, mass=True),
        # the offload-heavy 8B-like shape with its whole cache on the GPU, accumulating
        attention("decode 8B mass", "bf16", 32, 32, 8, 128, 65536, mass=True),
        # one long request alone
        attention("decode one long", "bf16", 1, 32, 8, 128, 131071),
        # eight drafted tokens of four requests verified in one call
        attention("verify 8 tokens", "bf16", 4, 32, 8, 128, 8200, queries=8),
        # the last tokens of a prompt look back over it, so that the first eviction has weights to go by
        attention("observe prompt mass", "bf16", 2, 32, 8, 128, 16384, queries=32, mass=True),
        # the new token of each of 32 requests
        append("append token 8B", "bf16", 32, 32, 8, 128, 1),
        # the prompts of four requests
        append("append prompt 8B", "bf16", 4, 32, 8, 128, 8192),
        # prompts of unequal, odd lengths in fp32
        append("append ragged f32", "f32", 3, 8, 2, 64, 1999, ragged=True),
        # one block too many in every unit: what a generation step meets every 64 tokens
        {"name": "evict one block", "op": "evict", "batch": 32, "hkv": 8, "blocks": 129, "budget": 128, "recent": 8},
        # a long prompt cut to its budget
        {"name": "evict prompt", "op": "evict", "batch": 32, "hkv": 8, "blocks": 1024, "budget": 64, "recent": 8},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["attention", "attention", "append", "evict"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 6, 8])
    d = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    batch = log(1, 32)
    if op == "attention":
        queries = rng.choice([1, 1, 1, rng.randint(2, 32)])
        most = min(131072, (1 << 29) // (batch * hkv * d * max(1, queries * hq // hkv // 8)))
        return {"op": op, "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d, "ctx": log(48, max(64, most)),
                "queries": queries, "ragged": rng.random() < 0.5, "mass": rng.random() < 0.5}
    if op == "append":
        most = min(16384, (1 << 25) // (batch * hkv * d))
        return {"op": op, "dtype": dtype, "batch": batch, "hq": hq, "hkv": hkv, "d": d,
                "tokens": 1 if rng.random() < 0.3 else log(2, max(4, most)), "ragged": rng.random() < 0.5}
    blocks = log(4, 2048)
    budget = rng.randint(2, blocks)
    return {"op": op, "batch": batch, "hkv": hkv, "blocks": blocks, "budget": budget,
            "recent": rng.randint(0, min(16, budget))}


# ---- what every part shares: lengths and sizes of a case ----------------------------------------------------------
def _lengths(case, most):
    """Tokens of each request: all `most`, or spread over 1..most."""
    n = case["batch"]
    if not case["ragged"]:
        return [most] * n
    return [max(1, most * ((5 * b) % n + 1) // n - 13 * b % 61) for b in range(n)]


def _unit_bytes(d):
    return -(-(2 * B * d + 4 * B + 8) // 32) * 32


def _elt(case):
    return 4 if case["dtype"] == "f32" else 2


def work(case):
    if case["op"] == "evict":
        n = case["batch"] * case["hkv"] * case["blocks"]
        return {"bytes": 16.0 * n, "flops": 0.0}
    d, hkv, elt = case["d"], case["hkv"], _elt(case)
    if case["op"] == "append":
        new = sum(_lengths(case, case["tokens"]))
        if case["tokens"] == 1:
            full = sum(_token_lens(case)[b] % B == B - 1 for b in range(case["batch"]))
            kept = new * (2 * d * elt + 4) + full * (B * (2 * d * elt + 4 + 2 * d + 4) + 8)
        else:
            full = sum(n // B for n in _lengths(case, case["tokens"]))
            kept = full * (B * (2 * d + 4) + 8) + sum(n % B for n in _lengths(case, case["tokens"])) * (2 * d * elt + 4)
        return {"bytes": float(hkv * (new * (2 * d * elt + 4) + kept)), "flops": float(2 * hkv * new * 2 * d)}
    lens = _lengths(case, case["ctx"])
    rows = case["batch"] * case["queries"] * case["hq"]
    full, tail = sum(n // B for n in lens), sum(n % B for n in lens)
    nbytes = hkv * (full * (B * (2 * d + 4) + 8 + 4) + tail * (2 * d * elt + 4)) + rows * (2 * d * elt + 4)
    if case["mass"]:
        nbytes += hkv * sum(-(-n // B) for n in lens) * 8
    return {"bytes": float(nbytes), "flops": float(4 * d * case["queries"] * case["hq"] * sum(lens))}


def _token_lens(case):
    """Lengths before a single token is appended: every 4th request completes a block."""
    return [4096 + 64 * b + (63 if b % 4 == 0 else 17 * b % 63) for b in range(case["batch"])]


# ---- inputs --------------------------------------------------------------------------------------------------------
def _codes(x, live):
    """Codes and scales of blocks x [..., 64, d] whose tokens count where live [..., 64]."""
    x = torch.where(live[..., None], x, 0.0)
    scale = x.abs().amax((-1, -2)) / 448
    return (x / scale.clamp(min=1e-30)[..., None, None]).clamp(-448, 448).to(E4M3), scale


def _image(k8, v8, e, ks, vs):
    """Block units from codes [n][64][d], logits [n][64] and scales [n]: the layout that the header documents."""
    n, d = k8.shape[0], k8.shape[-1]
    j = d // 32
    k = k8.view(torch.uint8).reshape(n, 4, 4, 2, 2, j, 2, 4, 4).permute(0, 1, 5, 2, 4, 7, 6, 3, 8)
    v = v8.view(torch.uint8).reshape(n, 4, 4, 4, j, 2, 2, 8).permute(0, 1, 4, 7, 2, 5, 6, 3)
    img = torch.zeros(n, _unit_bytes(d), dtype=torch.uint8, device=k8.device)
    body = img[:, : 2 * B * d].view(n, 4, 2, 16 * d)
    body[:, :, 0] = k.reshape(n, 4, 16 * d)
    body[:, :, 1] = v.reshape(n, 4, 16 * d)
    img[:, 2 * B * d : 2 * B * d + 4 * B] = e.contiguous().view(torch.uint8)
    img[:, 2 * B * d + 4 * B : 2 * B * d + 4 * B + 8] = torch.stack([ks, vs], 1).contiguous().view(torch.uint8)
    return img


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


def _per_unit(case, per_request):
    return torch.tensor(per_request, dtype=torch.int32, device="cuda").repeat_interleave(case["hkv"]).contiguous()


def _config(case):
    import trainable_sparse_attention_decode_gb300 as nosa
    return nosa.nosa_config(case["batch"], case.get("hq", case["hkv"]), case["hkv"], case.get("d", 128), case.get("dtype", "bf16"),
                            1, 0, 64)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    U = case["batch"] * case["hkv"]
    if case["op"] == "evict":
        n, extra = case["blocks"], 2  # the tail's entry and a spare one
        s["tab"] = torch.randperm(U * (n + extra), generator=g, device="cuda").to(torch.int32).view(U, n + extra)
        # accumulated weights: most blocks little, a few much; exact ties among the least
        m = torch.exp(2 * _normal(g, U, n + extra)).mul(64).round().div(64)
        s["mass"] = torch.where(torch.arange(n + extra, device="cuda") <= n, m, 0.0).contiguous()
        s["lens"] = torch.full((U,), n * B + 5, dtype=torch.int32, device="cuda")
        return s
    d, dtype = case["d"], TYPES[case["dtype"]]
    tb = _tail_bytes(d, _elt(case))
    s["tail"] = torch.zeros(U, tb, dtype=torch.uint8, device="cuda")
    tk, tv, te = _tail_parts(s["tail"], d, dtype)
    if case["op"] == "append":
        b, n, hkv = case["batch"], case["tokens"], case["hkv"]
        old = _token_lens(case) if n == 1 else [0] * b
        s["lens"] = _per_unit(case, old)
        if n == 1:  # the tails hold tokens already
            tk.copy_(_normal(g, *tk.shape))
            tv.copy_(_normal(g, *tv.shape))
            te.copy_(_logits(g, *te.shape))
        # one unit for each block that the call may complete; the entries before them are not this call's
        new = max(1, n // B)
        first = max(old) // B
        s["tab"] = torch.full((U, first + new + 1), -1, dtype=torch.int32, device="cuda")
        at = (s["lens"] // B)[:, None].long() + torch.arange(new, device="cuda")
        s["tab"].scatter_(1, at, torch.randperm(U * new, generator=g, device="cuda").to(torch.int32).view(U, new))
        s["units"] = torch.zeros(U * new, _unit_bytes(d), dtype=torch.uint8, device="cuda")
        s["k"] = (_normal(g, b, n, hkv, d) + 0.5 * _normal(g, b, 1, hkv, d)).to(dtype)
        s["v"] = _normal(g, b, n, hkv, d).to(dtype)
        s["e"] = _logits(g, b, n, hkv)
        s["n_new"] = torch.tensor(_lengths(case, n), dtype=torch.int32, device="cuda") if case["ragged"] else None
        s["lens_out"] = torch.empty_like(s["lens"])
        return s
    lens = _lengths(case, case["ctx"])
    s["lens"] = _per_unit(case, lens)
    tk.copy_(_normal(g, *tk.shape))
    tv.copy_(_normal(g, *tv.shape))
    te.copy_(_logits(g, *te.shape))
    blocks = [n // B for n in lens for _ in range(case["hkv"])]
    cap = max(-(-max(lens) // B), 1)
    total = sum(blocks)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    count = torch.tensor(blocks, device="cuda")
    at = torch.arange(cap, device="cuda")[None] + (count.cumsum(0) - count)[:, None]
    s["tab"] = torch.where(torch.arange(cap, device="cuda")[None] < count[:, None], perm[at.clamp(max=max(total - 1, 0))] if total else -1, -1)
    s["tab"] = s["tab"].to(torch.int32).contiguous()
    s["k8"] = torch.empty(total, B, d, dtype=E4M3, device="cuda")
    s["v8"] = torch.empty(total, B, d, dtype=E4M3, device="cuda")
    s["e"] = _logits(g, total, B)
    s["scales"] = torch.empty(total, 2, device="cuda")
    s["units"] = torch.empty(total, _unit_bytes(d), dtype=torch.uint8, device="cuda")
    for i in range(0, total, 1 << 15):  # a part at a time, so that the fp32 values need little room
        p = slice(i, min(total, i + (1 << 15)))
        m = p.stop - p.start
        live = s["e"][p] > -math.inf
        s["k8"][p], s["scales"][p, 0] = _codes(_normal(g, m, 1, d) + 0.5 * _normal(g, m, B, d), live)
        s["v8"][p], s["scales"][p, 1] = _codes(_normal(g, m, B, d), live)
        s["units"][p] = _image(s["k8"][p], s["v8"][p], s["e"][p], s["scales"][p, 0], s["scales"][p, 1])
    s["q"] = _normal(g, case["batch"], case["queries"], case["hq"], d).to(dtype)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(s["q"].shape[:3], device="cuda")
    s["mass"] = torch.rand(U, cap, generator=g, device="cuda") if case["mass"] else None
    return s


def _plan(s, make):
    """The configuration and workspace that a program keeps: made by the first call on a state."""
    if "plan" not in s:
        s["plan"] = make()
    return s["plan"]


DECAY = 0.96875


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    return {"attention": _attention, "append": _append, "evict": _evict}[s["case"]["op"]](s)


def _attention(s):
    case = s["case"]
    result = {"out": s["out"], "lse": s["lse"]}
    if s["mass"] is not None:
        result["mass"] = s["mass"]
    if own:
        import trainable_sparse_attention_decode_gb300 as nosa
        cfg, ws = _plan(s, lambda: (c := _config(case), torch.empty(
            nosa.nosa_quant_attention_workspace_bytes(c, s["tab"].shape[1], case["queries"], case["mass"]),
            dtype=torch.uint8, device="cuda")))
        nosa.nosa_quant_attention(cfg, s["units"], s["tab"], s["tail"], s["lens"], s["q"], s["out"], lse=s["lse"],
                                  mass=s["mass"], decay=DECAY, workspace=ws)
        return result
    b, T, hq, hkv, d = case["batch"], case["queries"], case["hq"], case["hkv"], case["d"]
    U, G, R = b * hkv, hq // hkv, T * hq // hkv
    cap = s["tab"].shape[1]
    q = s["q"].float().view(b, T, hkv, G, d).transpose(1, 2).reshape(U, R, d) / math.sqrt(d)
    # the positions of the full blocks, and of the tails
    lens = s["lens"].long()
    full = lens // B * B
    sees = (lens[:, None] - T + 1 + torch.arange(T, device="cuda")).repeat_interleave(G, 1)[..., None]  # [U][R][1]
    pos = torch.arange(cap * B, device="cuda")
    tpos = full[:, None, None] + torch.arange(B, device="cuda")
    tk, tv, te = _tail_parts(s["tail"], d, TYPES[case["dtype"]])
    tk = tk.transpose(1, 2).reshape(U, B, d).float()
    tlive = tpos < torch.minimum(sees, lens[:, None, None])
    tl = torch.where(tlive, q @ tk.transpose(1, 2) + te[:, None], -math.inf)
    logits = [tl]
    if s["k8"].shape[0]:
        tab = s["tab"].clamp(min=0).long()
        k = s["k8"].view(torch.uint8)[tab].view(E4M3).float().mul_(s["scales"][tab][..., 0][..., None, None])
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
        v = s["v8"].view(torch.uint8)[tab].view(E4M3).float().mul_(s["scales"][tab][..., 1][..., None, None])
        o = o + w[1] @ v.view(U, cap * B, d)
    mass.scatter_add_(1, (lens // B)[:, None], w[0].sum((1, 2))[:, None])
    heads = lambda x: x.view(b, hkv, T, G, -1).transpose(1, 2).reshape(b, T, hq, -1)  # noqa: E731
    s["out"].copy_(heads(o))
    s["lse"].copy_(heads(m + torch.log(z))[..., 0])
    if s["mass"] is not None:
        s["mass"].mul_(DECAY).add_(mass[:, :cap])
    return result


def _append(s):
    case = s["case"]
    d, dtype = case["d"], TYPES[case["dtype"]]
    if own:
        import trainable_sparse_attention_decode_gb300 as nosa
        cfg = _plan(s, lambda: _config(case))
        nosa.nosa_quant_append(cfg, s["k"], s["v"], s["e"], s["units"], s["tab"], s["tail"], s["lens"], s["lens_out"],
                               n_new=s["n_new"])
    else:
        b, n, hkv = case["batch"], case["tokens"], case["hkv"]
        U = b * hkv
        lens = s["lens"].long()
        new = s["n_new"].long().repeat_interleave(hkv) if s["n_new"] is not None else torch.full_like(lens, n)
        rows = lambda x: x.transpose(1, 2).reshape(U, n, -1)  # noqa: E731
        k, v, e = rows(s["k"]), rows(s["v"]), rows(s["e"][..., None])[..., 0]
        tk, tv, te = _tail_parts(s["tail"], d, dtype)
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
        live = e > -math.inf
        k8, ks = _codes(k[:, :blocks].float(), live[:, :blocks])
        v8, vs = _codes(v[:, :blocks].float(), live[:, :blocks])
        image = _image(k8.reshape(-1, B, d), v8.reshape(-1, B, d), e[:, :blocks].reshape(-1, B), ks.reshape(-1), vs.reshape(-1))
        done = ((lens % B + new) // B)[:, None]  # blocks completed
        j = torch.arange(blocks, device="cuda")
        to = s["tab"].gather(1, ((lens // B)[:, None] + j).clamp(max=s["tab"].shape[1] - 1)).long()
        to = torch.where(j < done, to, s["units"].shape[0])
        wide = torch.cat([s["units"], s["units"][:1]])  # one more row takes what is not stored
        wide[to.reshape(-1)] = image
        s["units"].copy_(wide[:-1])
        # what is left becomes the tails; rows behind them stay
        left = (lens % B + new - done[:, 0] * B)[:, None]
        r = torch.arange(B, device="cuda")
        take = lambda x: x.gather(1, done.view(U, 1, *[1] * (x.ndim - 2)).expand(U, 1, *x.shape[2:]))[:, 0]  # noqa: E731
        keep = r < left
        tk.copy_(torch.where(keep[:, None, :, None], take(k).view(U, B, *(tk.shape[1], tk.shape[3])).transpose(1, 2), tk))
        tv.copy_(torch.where(keep[..., None], take(v), tv))
        te.copy_(torch.where(keep, take(e), te))
        s["lens_out"].copy_(s["lens"] + new.to(torch.int32))
    tk, tv, te = _tail_parts(s["tail"], d, dtype)
    u = s["units"]
    return {"codes": u[:, : 2 * B * d].view(E4M3), "scales": u[:, 2 * B * d + 4 * B : 2 * B * d + 4 * B + 8].view(torch.float32),
            "logits": u[:, 2 * B * d : 2 * B * d + 4 * B].view(torch.float32), "tail_k": tk, "tail_v": tv, "tail_e": te,
            "lens": s["lens_out"]}


def _evict(s):
    case = s["case"]
    if own:
        import trainable_sparse_attention_decode_gb300 as nosa
        cfg, res = _plan(s, lambda: (_config(case), {"tab": torch.empty_like(s["tab"]), "mass": torch.empty_like(s["mass"]),
                                                     "lens": torch.empty_like(s["lens"]), "order": torch.empty_like(s["tab"])}))
        nosa.nosa_quant_evict(cfg, case["budget"], case["recent"], s["tab"], s["mass"], s["lens"], tab_out=res["tab"],
                              mass_out=res["mass"], lens_out=res["lens"], order=res["order"])
        return res
    tab, mass = s["tab"], s["mass"]
    cap = tab.shape[1]
    full = (s["lens"] // B).long()[:, None]
    j = torch.arange(cap, device="cuda")[None]
    over = (full - case["budget"]).clamp(min=0)
    # the newest first, then by weight, ties by index; what is no full block last
    rank = torch.where(j >= full, -math.inf, torch.where(j >= full - case["recent"], math.inf, mass))
    place = torch.sort(rank, dim=1, descending=True, stable=True).indices.argsort(1)
    gone = (place >= full - over) & (j < full) & (over > 0)
    order = torch.sort((gone | (j >= full)).long() + (j >= full).long(), dim=1, stable=True).indices
    at = full - over  # where the tail's weight goes
    moved = torch.where(j < at, mass.gather(1, order), torch.where(j == at, mass.gather(1, full.clamp(max=cap - 1)), 0.0))
    moved = torch.where((over > 0) & (j <= full) | (j < at), moved, mass)
    return {"tab": tab.gather(1, order), "mass": moved, "lens": s["lens"] - (over[:, 0] * B).to(torch.int32),
            "order": order.to(torch.int32)}


# ---- the definition in 64 bits ------------------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"attention": _exact_attention, "append": _exact_append, "evict": _exact_evict}[case["op"]](case, s)


def _exact_attention(case, s):
    T, hq, hkv, d = case["queries"], case["hq"], case["hkv"], case["d"]
    G = hq // hkv
    f64 = torch.float64
    out = torch.zeros(s["q"].shape, dtype=f64, device="cuda")
    lse = torch.full(s["lse"].shape, -math.inf, dtype=f64, device="cuda")
    mass = None if s["mass"] is None else s["mass"].to(f64) * DECAY
    tk, tv, te = _tail_parts(s["tail"], d, TYPES[case["dtype"]])
    lens = s["lens"].tolist()
    for u, n in enumerate(lens):
        b, h = u // hkv, u % hkv
        nb, nt = n // B, n % B
        ids = s["tab"][u, :nb].long()
        sk, sv = s["scales"][ids].to(f64).unbind(1)
        keys = (s["k8"].view(torch.uint8)[ids].view(E4M3).to(f64) * sk.view(-1, 1, 1)).view(nb * B, d)
        vals = (s["v8"].view(torch.uint8)[ids].view(E4M3).to(f64) * sv.view(-1, 1, 1)).view(nb * B, d)
        keys = torch.cat([keys, tk[u].to(f64).permute(1, 0, 2).reshape(B, d)[:nt]])
        vals = torch.cat([vals, tv[u, :nt].to(f64)])
        bias = torch.cat([s["e"][ids].view(-1), te[u, :nt]]).to(f64)
        qs = s["q"][b, :, h * G : (h + 1) * G].to(f64).reshape(T * G, d)
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


def _exact_append(case, s):
    d, hkv, dtype = case["d"], case["hkv"], TYPES[case["dtype"]]
    f64 = torch.float64
    U = case["batch"] * hkv
    tk, tv, te = [x.clone() for x in _tail_parts(s["tail"], d, dtype)]
    lens = s["lens"].tolist()
    new = s["n_new"].tolist() if s["n_new"] is not None else [case["tokens"]] * case["batch"]
    units = s["units"].shape[0]
    codes = torch.zeros(units, 2 * B * d, dtype=f64, device="cuda")
    scales = torch.zeros(units, 2, dtype=f64, device="cuda")
    logits = torch.zeros(units, B, dtype=f64, device="cuda")
    after = []
    # where code (token, dim) of the keys and of the values stands in a unit
    t, x = torch.arange(B, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    w, tt = t // 16, t % 16
    g, half = 2 * (tt // 4) + tt % 2, tt % 4 // 2
    k_at = w * 32 * d + (x // 32 * 32 + g * 4 + x % 16 // 4) * 16 + (x % 32 // 16 * 2 + half) * 4 + x % 4
    v_at = w * 32 * d + 16 * d + (x // 32 * 32 + x % 8 * 4 + tt // 4) * 16 + (x % 32 // 16 * 2 + x % 16 // 8) * 4 + tt % 4
    for u in range(U):
        b, h = u // hkv, u % hkv
        n0, n1 = lens[u], lens[u] + new[b]
        after.append(n1)
        old = n0 % B
        k = torch.cat([tk[u].permute(1, 0, 2).reshape(B, d)[:old], s["k"][b, : new[b], h]])
        v = torch.cat([tv[u, :old], s["v"][b, : new[b], h]])
        e = torch.cat([te[u, :old], s["e"][b, : new[b], h]])
        done = k.shape[0] // B
        if done:
            to = s["tab"][u, n0 // B : n0 // B + done].long()
            eb = e[: done * B].view(done, B)
            logits[to] = eb.to(f64)
            for i, (src, at) in enumerate(((k, k_at), (v, v_at))):
                y = src[: done * B].to(f64).view(done, B, d).masked_fill(eb.isneginf()[..., None], 0.0)
                sc = y.abs().flatten(1).max(1).values / 448
                scales[to, i] = sc
                part = codes[to]
                part[:, at.reshape(-1)] = (y / sc.view(-1, 1, 1)).reshape(done, -1)
                codes[to] = part
        left = k.shape[0] - done * B
        first = old if not done else 0  # a tail that goes on keeps its rows
        if left > first:
            rows = slice(done * B + first, done * B + left)
            tk[u][:, first:left] = k[rows].view(left - first, tk.shape[1], tk.shape[3]).transpose(0, 1)
            tv[u][first:left] = v[rows]
            te[u][first:left] = e[rows]
    return {"codes": codes, "scales": scales, "logits": logits, "tail_k": tk.to(f64), "tail_v": tv.to(f64), "tail_e": te.to(f64),
            "lens": torch.tensor(after, dtype=torch.int32, device="cuda")}


def _exact_evict(case, s):
    tab, mass, lens = s["tab"].tolist(), s["mass"].tolist(), s["lens"].tolist()
    out_tab, out_mass, out_lens, out_order = [], [], [], []
    for row, m, n in zip(tab, mass, lens):
        full = n // B
        over = max(0, full - case["budget"])
        old = range(full - min(case["recent"], full))
        gone = set(sorted(old, key=lambda i: (m[i], -i))[:over])
        order = [i for i in range(full) if i not in gone] + sorted(gone) + list(range(full, len(row)))
        moved = [m[i] for i in order[: full - over]]
        if over:
            moved += [m[full]] + [0.0] * over
        moved += m[len(moved):]
        out_tab.append([row[i] for i in order])
        out_mass.append(moved)
        out_lens.append(n - over * B)
        out_order.append(order)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    return {"tab": torch.tensor(out_tab, **i32), "mass": torch.tensor(out_mass, dtype=torch.float64, device="cuda"),
            "lens": torch.tensor(out_lens, **i32), "order": torch.tensor(out_order, **i32)}
