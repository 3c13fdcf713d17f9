"""Cases and plain forms of the paged-cache operators around the sparse layer.

Three operators that a serving step runs one after the other in a layer with rotary positions:

  rope    rotary positions on the queries (and keys) of a call's tokens
  append  the new tokens' keys, rotated on the way, and values into a paged cache, and the rotation of their queries
  attn    attention of each sequence's newest tokens (one, a few or a long chunk) over its paged cache

``run`` computes them in elementary torch operations, or, where ``own`` is set, by the framework's entry points.
A cache is [pages, 64, heads, width]; position p of sequence b lies in page block_table[b, p // 64].  Caches in 8 bits
hold e4m3 codes of value * scale.
"""
import math
import random

import torch

own = False

PAGE = 64
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
K_SCALE, V_SCALE = 32.0, 64.0  # of the e4m3 caches: unit-normal values use the type's range without saturating


# ---- the cases -------------------------------------------------------------------------------------------------


def listed():
    return [
        # one decode step's queries of the sparse layer: 8 sequences, 128 heads of 512 + 64, far positions; latency
        {"name": "rope_step_8", "op": "rope", "T": 8, "H": 128, "Hk": 0, "D": 576, "dim": 64, "offset": 512,
         "interleaved": True, "inverse": False, "yarn": 1.0, "max_pos": 131072, "type": "bf16", "fused": False},
        # a long prompt's queries and keys of the local layers (64 heads x 128), the whole head rotated; bandwidth
        {"name": "rope_chunk_16384", "op": "rope", "T": 16384, "H": 64, "Hk": 64, "D": 128, "dim": 128, "offset": 0,
         "interleaved": False, "inverse": False, "yarn": 1.0, "max_pos": 32768, "type": "bf16", "fused": True},
        # keys and queries of a million-token context turned back to where they were (the transpose, a gradient's
        # pass too), half of the head rotated, frequencies stretched for the long context, an odd number of tokens
        {"name": "rope_back_1001", "op": "rope", "T": 1001, "H": 32, "Hk": 8, "D": 128, "dim": 64, "offset": 0,
         "interleaved": False, "inverse": True, "yarn": 32.0, "max_pos": 1048576, "type": "f16", "fused": True},
        # one decode step of the hybrid's 64 sequences in a layer of 64 query and 8 key heads; latency
        {"name": "append_step_64", "op": "append", "n": 64, "B": 64, "min_len": 4096, "max_len": 65536, "pages": 512,
         "H": 64, "Hkv": 8, "Dk": 128, "Dv": 128, "dim": 128, "offset": 0, "interleaved": False, "yarn": 1.0,
         "type": "bf16", "cache": "bf16", "ragged": 1},
        # a prompt's latent rows of the sparse layer: 512 elements as they are, 64 rotated, no values of their own
        {"name": "append_latent_32768", "op": "append", "n": 32768, "B": 8, "min_len": 4096, "max_len": 4096,
         "pages": 768, "H": 0, "Hkv": 1, "Dk": 576, "Dv": 0, "dim": 64, "offset": 512, "interleaved": True,
         "yarn": 1.0, "type": "bf16", "cache": "bf16", "ragged": 2},
        # chunks of several prompts into an 8-bit cache, an odd number of tokens
        {"name": "append_fp8_4099", "op": "append", "n": 4099, "B": 5, "min_len": 1000, "max_len": 20000, "pages": 1100,
         "H": 64, "Hkv": 8, "Dk": 128, "Dv": 128, "dim": 64, "offset": 0, "interleaved": False, "yarn": 4.0,
         "type": "bf16", "cache": "e4m3", "ragged": 3},
        # one user, one token: what a single stream waits for in each full-attention layer
        {"name": "attn_single_4097", "op": "attn", "B": 1, "min_q": 1, "max_q": 1, "min_len": 4097, "max_len": 4097,
         "H": 64, "Hkv": 8, "D": 128, "window": 0, "type": "bf16", "cache": "bf16", "lse": False, "ragged": 4},
        # the hybrid's decode batch in a full-attention layer: every sequence's whole history is read
        {"name": "attn_decode_64", "op": "attn", "B": 64, "min_q": 1, "max_q": 1, "min_len": 4096, "max_len": 65536,
         "H": 64, "Hkv": 8, "D": 128, "window": 0, "type": "bf16", "cache": "bf16", "lse": False, "ragged": 5},
        # the same step over an 8-bit cache, fewer and shorter sequences, and the log-sum-exp for a later merge
        {"name": "attn_decode_fp8_33", "op": "attn", "B": 33, "min_q": 1, "max_q": 1, "min_len": 1000,
         "max_len": 40000, "H": 64, "Hkv": 8, "D": 128, "window": 0, "type": "bf16", "cache": "e4m3", "lse": True,
         "ragged": 6},
        # four draft tokens a sequence over long contexts
        {"name": "attn_drafts_8x4", "op": "attn", "B": 8, "min_q": 4, "max_q": 4, "min_len": 131072,
         "max_len": 131072, "H": 64, "Hkv": 8, "D": 128, "window": 0, "type": "bf16", "cache": "bf16", "lse": False,
         "ragged": 7},
        # chunks of prompts in the hybrid's local layers: 64 heads of their own keys, window 128
        {"name": "attn_local_8", "op": "attn", "B": 8, "min_q": 257, "max_q": 2048, "min_len": 2048, "max_len": 4096,
         "H": 64, "Hkv": 64, "D": 128, "window": 128, "type": "bf16", "cache": "bf16", "lse": False, "ragged": 8},
        # the next 4096 tokens of a long prompt over the 32768 positions that it then has
        {"name": "attn_chunk_4096", "op": "attn", "B": 1, "min_q": 4096, "max_q": 4096, "min_len": 32768,
         "max_len": 32768, "H": 32, "Hkv": 4, "D": 128, "window": 0, "type": "bf16", "cache": "bf16", "lse": True,
         "ragged": 9},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["rope", "append", "attn", "attn"])
    t = rng.choice(["bf16", "bf16", "f16"])
    seed = rng.randrange(1 << 30)
    if kind == "rope":
        D = rng.choice([64, 96, 128, 256, 576])
        dim = 64 if D == 576 else rng.choice([D, D // 2, D // 4])
        T, H = _log_int(rng, 1, 8192), rng.choice([1, 5, 8, 16, 32, 64])
        return {"op": "rope", "T": T, "H": H, "Hk": rng.choice([0, 1, 8]), "D": D, "dim": dim,
                "offset": rng.choice([0, D - dim]), "interleaved": rng.random() < 0.5, "inverse": rng.random() < 0.3,
                "yarn": rng.choice([1.0, 4.0, 32.0]), "max_pos": _log_int(rng, 4096, 1048576), "type": t,
                "fused": rng.random() < 0.5}
    if kind == "append":
        latent = rng.random() < 0.25
        n, B = _log_int(rng, 1, 16384), _log_int(rng, 1, 64)
        D = 576 if latent else rng.choice([64, 128])
        dim = 64 if latent else rng.choice([D, D // 2])
        lo = max(256, -(-n // B))
        return {"op": "append", "n": n, "B": B, "min_len": lo, "max_len": lo + _log_int(rng, 1, 8192),
                "pages": -(-n // PAGE) + 3 * B + 5, "H": rng.choice([0, 16, 64]), "Hkv": 1 if latent else rng.choice([1, 2, 8]),
                "Dk": D, "Dv": 0 if latent else D, "dim": dim, "offset": D - dim if latent else 0,
                "interleaved": rng.random() < 0.5, "yarn": rng.choice([1.0, 16.0]), "type": t,
                "cache": t if latent else rng.choice([t, "e4m3"]), "ragged": seed}
    Hkv, G, D = rng.choice([1, 2, 8]), rng.choice([1, 4, 5, 8, 16]), rng.choice([64, 128, 128])
    cache, window = rng.choice([t, t, "e4m3"]), rng.choice([0, 0, 128, 1000])
    if rng.random() < 0.5:  # one or a few tokens of each of many sequences
        B, q = _log_int(rng, 1, 64), rng.choice([1, 1, 1, 2, 5])
        lo = _log_int(rng, 8, 4096)
        return {"op": "attn", "B": B, "min_q": q, "max_q": q, "min_len": lo, "max_len": _log_int(rng, lo, 32768), "H": Hkv * G,
                "Hkv": Hkv, "D": D, "window": window, "type": t, "cache": cache, "lse": rng.random() < 0.5, "ragged": seed}
    B, q, G = rng.choice([1, 2, 3]), _log_int(rng, 33, 2000), min(G, 8)
    lo = q + _log_int(rng, 1, 2000)
    return {"op": "attn", "B": B, "min_q": max(1, q // 4), "max_q": q, "min_len": lo, "max_len": lo + _log_int(rng, 1, 4000),
            "H": Hkv * G, "Hkv": Hkv, "D": D, "window": window, "type": t, "cache": cache, "lse": rng.random() < 0.5,
            "ragged": seed}


def _lengths(case):
    """Every sequence's length and number of newest tokens: a matter of the case alone."""
    r = random.Random(case["ragged"])
    lens = [r.randint(case["min_len"], case["max_len"]) for _ in range(case["B"])]
    if case["op"] == "append":  # the call's n tokens, dealt out evenly: each sequence's last ones
        new = [case["n"] // case["B"] + (b < case["n"] % case["B"]) for b in range(case["B"])]
    else:
        new = [r.randint(case["min_q"], case["max_q"]) for _ in range(case["B"])]
    return [max(a, b) for a, b in zip(lens, new)], new


def _frequencies(case):
    """Radians a position of each pair, and the factor on cos and sin: base 10000, stretched for contexts `yarn` times
    as long as 4096 positions (slow pairs interpolated, fast ones kept, a ramp between)."""
    half, s = case["dim"] // 2, case["yarn"]
    plain = [10000.0 ** (-i / half) for i in range(half)]
    if s == 1.0:
        return plain, 1.0
    turn = lambda turns: half * math.log(4096 / (turns * 2 * math.pi)) / math.log(10000.0)  # noqa: E731
    lo, hi = max(math.floor(turn(32)), 0), min(math.ceil(turn(1)), case["dim"] - 1)
    ramp = [min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(half)]
    return [f * (1 - r) + f / s * r for f, r in zip(plain, ramp)], 0.1 * math.log(s) + 1.0


# ---- what a program has in hand before the call -------------------------------------------------------------------


def _heads(g, T, heads, D, dtype, fused):
    """The head groups of one projection's output: views of one fused buffer, or each its own."""
    if fused:
        buf = torch.randn(T, sum(heads), D, generator=g, device="cuda", dtype=torch.float32).to(dtype)
        return list(buf.split(heads, dim=1))
    return [torch.randn(T, h, D, generator=g, device="cuda", dtype=torch.float32).to(dtype) for h in heads]


def _cache(g, pages, heads, width, dtype, scale):
    c = torch.empty(pages, PAGE, heads, width, device="cuda", dtype=dtype)
    for i in range(0, pages, 1024):  # a piece at a time: the draws are in 32 bits
        part = c[i:i + 1024]
        x = torch.randn(part.shape, generator=g, device="cuda", dtype=torch.float32)
        part.copy_((x * scale if dtype == torch.float8_e4m3fn else x).to(dtype))
    return c


def _ints(values):
    return torch.tensor(values, device="cuda", dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = TYPES[case["type"]]
    s = {"case": case}
    if case["op"] in ("rope", "append"):
        freq, s["factor"] = _frequencies(case)
        s["inv_freq"] = torch.tensor(freq, device="cuda", dtype=torch.float64)
    if case["op"] == "rope":
        s["q"], s["k"], _ = _heads(g, case["T"], [case["H"], case["Hk"], case["Hk"]], case["D"], dtype, case["fused"])
        s["pos"] = torch.randint(0, case["max_pos"], (case["T"],), generator=g, device="cuda", dtype=torch.int32)
    else:
        lens, new = _lengths(case)
        blocks = -(-max(lens) // PAGE)
        width, heads = (case["Dk"], case["Hkv"]) if case["op"] == "append" else (case["D"], case["Hkv"])
        first = [(n - m) // PAGE if case["op"] == "append" else 0 for n, m in zip(lens, new)]  # an append needs no older page
        used = [-(-n // PAGE) - f for n, f in zip(lens, first)]
        pages = case["pages"] if case["op"] == "append" else sum(used) + 3
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table, at = torch.zeros(case["B"], blocks, device="cuda", dtype=torch.int32), 0
        for b, (f, u) in enumerate(zip(first, used)):
            table[b, f:f + u] = order[at:at + u]
            at += u
        s["lens"], s["table"], s["pages"] = _ints(lens), table, pages
        cache = TYPES[case["cache"]]
        s["k_cache"] = _cache(g, pages, heads, width, cache, K_SCALE)
        if case["op"] == "append":
            s["v_cache"] = _cache(g, pages, heads, case["Dv"], cache, V_SCALE) if case["Dv"] else None
            q, s["k"], v = _heads(g, case["n"], [case["H"], heads, heads if case["Dv"] else 0], width, dtype, False)
            s["q"], s["v"] = q if case["H"] else None, v if case["Dv"] else None
            s["tok_seq"] = _ints([b for b, m in enumerate(new) for _ in range(m)])
            s["tok_pos"] = _ints([n - m + i for n, m in zip(lens, new) for i in range(m)])
        else:
            s["v_cache"] = _cache(g, pages, heads, width, cache, V_SCALE)
            s["T"], s["max_q"], s["max_len"] = sum(new), max(new), max(lens)
            s["q"] = _heads(g, s["T"], [case["H"]], width, dtype, False)[0]
            s["q_start"] = _ints([sum(new[:b]) for b in range(case["B"] + 1)])
    if own:  # the views that a program makes once: frequencies, cache, page table, workspace
        from long_context_sparse_02_b200 import _lib
        if case["op"] != "attn":
            s["spec"] = _lib.rope_spec(s["inv_freq"], offset=case["offset"], interleaved=case["interleaved"],
                                       inverse=case.get("inverse", False), factor=s["factor"])
        if case["op"] != "rope":
            s["pg"] = _lib.paged(s["lens"], s["table"], s["pages"])
            s["cache"] = _lib.kv_cache(s["k_cache"], s["v_cache"], K_SCALE, V_SCALE)
        if case["op"] == "attn":
            s["ws"] = _lib.paged_attn_workspace(s["T"], case["H"], s["cache"], s["pg"], s["max_q"], s["max_len"],
                                                case["window"])
    return s


# ---- one pass --------------------------------------------------------------------------------------------------------


def _rotated(x, pos, s):
    """x [T, heads, D] rotated, in 32 bits; angles in 64 (positions reach a million)."""
    c = s["case"]
    angle = pos.double()[:, None, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["factor"]).float(), (angle.sin() * s["factor"]).float()
    if c.get("inverse"):
        sin = -sin
    y, half = x.float(), c["dim"] // 2
    part = y[..., c["offset"]:c["offset"] + c["dim"]]
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :half], part[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((y[..., :c["offset"]], turned, y[..., c["offset"] + c["dim"]:]), -1)


def _stored(x, dtype, scale):
    return (x.float() * scale).clamp(-448, 448).to(dtype) if dtype == torch.float8_e4m3fn else x.to(dtype)


def _plain_append(s):
    dtype = s["k_cache"].dtype
    page = s["table"][s["tok_seq"].long(), s["tok_pos"].long() // PAGE].long()
    row = s["tok_pos"].long() % PAGE
    bits = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
    s["k_cache"].view(bits)[page, row] = _stored(_rotated(s["k"], s["tok_pos"], s), dtype, K_SCALE).view(bits)
    if s["v"] is not None:
        s["v_cache"].view(bits)[page, row] = _stored(s["v"], dtype, V_SCALE).view(bits)
    q = _rotated(s["q"], s["tok_pos"], s).to(s["q"].dtype) if s["q"] is not None else None
    return q


def _plain_attn(s):
    c, q = s["case"], s["q"]
    B, Hkv, G, D = c["B"], c["Hkv"], c["H"] // c["Hkv"], c["D"]
    n, start, lens = s["max_q"], s["q_start"].long(), s["lens"].long()
    new = start[1:] - start[:-1]
    token = torch.arange(n, device="cuda")
    real = token < new[:, None]  # [B, n]: sequences with fewer new tokens than the most are padded
    rows = torch.where(real, start[:-1, None] + token, 0)
    qp = q[rows].float().reshape(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    eight = s["k_cache"].dtype == torch.float8_e4m3fn
    table = s["table"].long()

    def history(cache, scale):  # [B, Hkv, positions, D]
        x = cache.view(torch.uint8)[table].view(cache.dtype) if eight else cache[table]
        x = x.reshape(B, -1, Hkv, D).transpose(1, 2).float()
        return x / scale if eight else x

    keys = history(s["k_cache"], K_SCALE)
    scores = (qp @ keys.transpose(-1, -2)).view(B, Hkv, G, n, -1)
    del keys
    scores *= 1 / math.sqrt(D)
    at, pos = torch.arange(scores.shape[-1], device="cuda"), (lens - new)[:, None] + token
    seen = at <= pos[..., None]
    if c["window"]:
        seen &= at > pos[..., None] - c["window"]
    scores.masked_fill_(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, G * n, -1) @ history(s["v_cache"], V_SCALE)).view(B, Hkv, G, n, D) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(B, n, c["H"], D)[real].to(q.dtype)
    if not c["lse"]:
        return out
    return out, (top + total.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, c["H"])[real]


def run(s):
    c = s["case"]
    if c["op"] == "rope":
        if own:
            from long_context_sparse_02_b200 import _lib
            q, k = _lib.rope(s["q"], s["pos"], s["spec"], k=s["k"] if c["Hk"] else None)
        else:
            q = _rotated(s["q"], s["pos"], s).to(s["q"].dtype)
            k = _rotated(s["k"], s["pos"], s).to(s["k"].dtype) if c["Hk"] else None
        return {"q": q, "k": k}
    if c["op"] == "append":
        if own:
            from long_context_sparse_02_b200 import _lib
            q = _lib.append_rope(s["k"], s["v"], s["tok_seq"], s["tok_pos"], s["pg"], s["cache"], s["spec"], q=s["q"])
        else:
            q = _plain_append(s)
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if own:
        from long_context_sparse_02_b200 import _lib
        return _lib.paged_attn(s["q"], s["cache"], s["pg"], s["q_start"], s["max_q"], s["max_len"], c["window"],
                               1 / math.sqrt(c["D"]), want_lse=c["lse"], ws=s["ws"])
    return _plain_attn(s)


# ---- the work of one pass ------------------------------------------------------------------------------------------------


def work(case):
    e = 2  # bf16 and fp16
    if case["op"] == "rope":
        heads = case["T"] * (case["H"] + case["Hk"])
        return {"bytes": 2 * heads * case["D"] * e + 4 * case["T"] + 4 * case["dim"], "flops": 3 * heads * case["dim"]}
    lens, new = _lengths(case)
    c = 1 if case["cache"] == "e4m3" else 2
    if case["op"] == "append":
        row = case["Hkv"] * (case["Dk"] + case["Dv"]) * (e + c) + 2 * case["H"] * case["Dk"] * e + 12
        return {"bytes": case["n"] * row, "flops": 3 * case["n"] * (case["H"] + case["Hkv"]) * case["dim"]}
    w, seen, read = case["window"], 0, 0
    for n, m in zip(lens, new):
        first = n - m  # the position of the first new token
        seen += sum(min(p + 1, w) for p in range(first, n)) if w else m * first + m * (m + 1) // 2
        read += min(n, w + m - 1) if w else n
    T = sum(new)
    return {"bytes": read * case["Hkv"] * case["D"] * 2 * c + 2 * T * case["H"] * case["D"] * e + 4 * case["lse"] * T * case["H"],
            "flops": 4 * seen * case["H"] * case["D"]}


# ---- the definition in 64 bits -----------------------------------------------------------------------------------------


def _turned64(x, pos, s):
    """Pairs as complex numbers, each times factor * e^(i angle)."""
    c = s["case"]
    z = x.double()
    lo, half = c["offset"], c["dim"] // 2
    step = 2 if c["interleaved"] else 1
    re = slice(lo, lo + c["dim"], 2) if step == 2 else slice(lo, lo + half)
    im = slice(lo + 1, lo + c["dim"], 2) if step == 2 else slice(lo + half, lo + c["dim"])
    angle = torch.outer(pos.double(), s["inv_freq"]) * (-1.0 if c.get("inverse") else 1.0)
    w = torch.complex(z[..., re].contiguous(), z[..., im].contiguous())
    w *= torch.polar(torch.full_like(angle, s["factor"]), angle)[:, None]
    z[..., re], z[..., im] = w.real, w.imag
    return z


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _turned64(s["q"], s["pos"], s), "k": _turned64(s["k"], s["pos"], s) if case["Hk"] else None}
    lens, new = _lengths(case)
    eight = case["cache"] == "e4m3"
    if case["op"] == "append":
        got = {"q": _turned64(s["q"], s["tok_pos"], s) if case["H"] else None}
        at = (s["table"].cpu(), s["tok_seq"].tolist(), s["tok_pos"].tolist())
        slot = torch.tensor([int(at[0][b, p // PAGE]) * PAGE + p % PAGE for b, p in zip(at[1], at[2])], device="cuda")
        for key, new_rows, scale in (("k_cache", _turned64(s["k"], s["tok_pos"], s), K_SCALE), ("v_cache", s["v"], V_SCALE)):
            if s[key] is None:
                got[key] = None
                continue
            whole = s[key].double().flatten(0, 1)
            x = new_rows.double()
            whole[slot] = torch.clamp(x * scale, -448.0, 448.0) if eight else x
            got[key] = whole.view(s[key].shape)
        return got
    G, D = case["H"] // case["Hkv"], case["D"]
    out = torch.empty(s["T"], case["H"], D, device="cuda", dtype=torch.float64)
    lse = torch.empty(s["T"], case["H"], device="cuda", dtype=torch.float64)
    t0 = 0
    for b, (n, m) in enumerate(zip(lens, new)):
        pages = s["table"][b, :-(-n // PAGE)].long()
        p = torch.arange(n - m, n, device="cuda")[:, None]
        x = torch.arange(n, device="cuda")[None]
        bad = (x > p) | ((x <= p - case["window"]) if case["window"] else False)
        for h in range(case["Hkv"]):
            k, v = (s[key][pages, :, h].double().reshape(-1, D)[:n] if not eight else
                    s[key].view(torch.uint8)[pages, :, h].view(TYPES["e4m3"]).double().reshape(-1, D)[:n] / scale
                    for key, scale in (("k_cache", K_SCALE), ("v_cache", V_SCALE)))
            for head in range(h * G, (h + 1) * G):
                logits = s["q"][t0:t0 + m, head].double() @ k.T / math.sqrt(D)
                logits[bad] = -math.inf
                lse[t0:t0 + m, head] = torch.logsumexp(logits, -1)
                out[t0:t0 + m, head] = torch.softmax(logits, -1) @ v
        t0 += m
    return (out, lse) if case["lse"] else out
