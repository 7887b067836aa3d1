"""The measured cases of the prompt side of the paged cache: writing a chunk's q, k and v
(norm, rotation, cache write), attending it over the pages, and reading pages back.

Each case is run either through the package's public calls (`own` true) or in its plain
form: elementary torch operations in 32 bits (64 for the angles of far positions), rounded
once at the end.
"""
import math
import random

import torch

own = False

BLOCK = 16
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one user's next token over a short chat: nothing but latency
        attend("attend_one_token", 1, (1, 1), (776, 776), 32, 8, 128),
        # speculated tokens of 24 running requests checked at once: few rows, long ragged contexts
        attend("attend_verify", 24, (3, 8), (1800, 12000), 32, 8, 128),
        # prompts of a batch of new requests, nothing cached yet, odd lengths
        attend("attend_prompts", 9, (257, 2048), (0, 0), 32, 8, 128),
        # a chunk of a long document late in its prefill: the largest products
        attend("attend_long_chunk", 1, (4096, 4096), (28672, 28672), 32, 8, 128),
        # chunks of four requests over an 8-bit cache, the wider query group
        attend("attend_e4m3_chunks", 4, (700, 1100), (3000, 9000), 64, 8, 128, e4m3=True),
        # a decoder's tokens over an encoder's states kept in pages: no causal mask, small heads
        attend("attend_cross", 16, (1, 448), (750, 1500), 8, 2, 64, causal=False, lse=True),
        # one decode step of 64 requests: norm, rotation and cache write
        write("write_step", 64, 32, 8, 128, norm=True, far=131072),
        # a prefill batch into an 8-bit cache
        write("write_prefill_e4m3", 8192, 32, 8, 128, norm=True, e4m3=True, far=32768),
        # small heads, a quarter of the head rotated in pairs, no norm, an odd count
        write("write_interleaved", 20011, 8, 2, 64, rot=16, interleaved=True, far=8192),
        # one request's pages handed to another machine
        gather("read_one", 1, (1000, 1000), 8, 128),
        # the pages of a decode batch read back
        gather("read_batch", 64, (512, 4096), 8, 128),
        # long 8-bit contexts read back dequantised
        gather("read_long_e4m3", 4, (32768, 70000), 8, 128, e4m3=True, fp32=True),
    ]


def attend(name, batch, new, past, hq, hkv, d, e4m3=False, causal=True, lse=False, shape_seed=1):
    return {"name": name, "kind": "attend", "batch": batch, "new_min": new[0], "new_max": new[1], "past_min": past[0],
            "past_max": past[1], "hq": hq, "hkv": hkv, "d": d, "e4m3": e4m3, "causal": causal, "lse": lse,
            "shape_seed": shape_seed}


def write(name, tokens, hq, hkv, d, norm=False, e4m3=False, rot=None, interleaved=False, far=8192, shape_seed=1):
    return {"name": name, "kind": "write", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "norm": norm, "e4m3": e4m3,
            "rot": d if rot is None else rot, "interleaved": interleaved, "far": far, "shape_seed": shape_seed}


def gather(name, batch, lens, hkv, d, e4m3=False, fp32=False, shape_seed=1):
    return {"name": name, "kind": "gather", "batch": batch, "len_min": lens[0], "len_max": lens[1], "hkv": hkv, "d": d,
            "e4m3": e4m3, "fp32": fp32, "shape_seed": shape_seed}


def spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    kind = rng.choice(("attend", "attend", "write", "gather"))
    hq, hkv, d = rng.choice(((32, 8, 128), (64, 8, 128), (8, 2, 64), (16, 16, 64), (16, 8, 128)))
    if kind == "write":
        c = write("", spread(rng, 1, 16384), hq, hkv, d, rng.random() < 0.5, rng.random() < 0.5,
                  rng.choice((16, d // 2, d)), rng.random() < 0.4, spread(rng, 2048, 1 << 20), seed)
    elif kind == "gather":
        batch = spread(rng, 1, 64)
        top = spread(rng, 16, min(32768, (1 << 18) // batch))
        c = gather("", batch, (rng.randint(0, top), top), hkv, d, rng.random() < 0.5, rng.random() < 0.5, seed)
    else:
        batch = spread(rng, 1, 24)
        past = spread(rng, 1, 16384) if rng.random() < 0.8 else 0
        room = (1 << 31) // (batch * hq)  # of score entries for a sequence, padded
        new = spread(rng, 1, 2048)
        while new > 1 and new * (past + new) > room:
            new = (new + 1) // 2
        causal = rng.random() < 0.8 or past < 2
        c = attend("", batch, (rng.randint(1, new), new), (rng.randint(0 if causal else 1, past), past) if past else (0, 0),
                   hq, hkv, d, rng.random() < 0.4, causal, rng.random() < 0.3, seed)
    del c["name"]
    return c


def lengths(case):
    """(new tokens, cached tokens among them) of every sequence of an attend case."""
    r = random.Random(case["shape_seed"])
    new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
    past = [r.randint(case["past_min"], case["past_max"]) for _ in range(case["batch"])]
    return new, [p + n for n, p in zip(new, past)] if case["causal"] else past


def spans(case):
    r = random.Random(case["shape_seed"])
    return [r.randint(case["len_min"], case["len_max"]) for _ in range(case["batch"])]


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def work(case):
    hkv, d, one = case["hkv"], case["d"], 1 if case["e4m3"] else 2
    if case["kind"] == "attend":
        new, ctx = lengths(case)
        pairs = sum(n * c - (n * (n - 1) // 2 if case["causal"] else 0) for n, c in zip(new, ctx))
        rows = sum(new) * case["hq"]
        return {"bytes": rows * d * 4 + sum(ctx) * hkv * d * 2 * one + (rows * 4 if case["lse"] else 0),
                "flops": 4 * d * case["hq"] * pairs}
    if case["kind"] == "write":
        t = case["tokens"]
        return {"bytes": t * d * (case["hq"] * 4 + hkv * 4 + hkv * 2 * one) + t * 12, "flops": t * d * (case["hq"] + hkv) * 8}
    rows = sum(spans(case))
    return {"bytes": rows * hkv * d * 2 * (one + (4 if case["fp32"] else 2)), "flops": rows * hkv * d * 2}


# ------------------------------------------------------------------ inputs

def pool(g, blocks, case):
    """A pool of random K and V (E4M3 codes with their scales, or bf16)."""
    shape = (blocks, BLOCK, case["hkv"], case["d"])
    k, v = (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16) for _ in range(2))
    if not case["e4m3"]:
        return k, v, None
    scales = torch.rand((2, case["hkv"]), generator=g, device=DEV) * 0.01 + 0.01
    k, v = ((x.float() / scales[i][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn) for i, x in enumerate((k, v)))
    return k, v, scales


def tables(g, lens):
    """Block tables of sequences of these lengths over a shuffled pool, and its blocks."""
    need = [max(1, (n + BLOCK - 1) // BLOCK) for n in lens]
    wide, total = max(need), sum(need)
    blocks = total + total // 10 + 4
    ids = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    at = torch.tensor(offsets(need)[:-1], device=DEV)[:, None] + torch.arange(wide, device=DEV)
    used = torch.arange(wide, device=DEV) < torch.tensor(need, device=DEV)[:, None]
    return torch.where(used, ids[at.clamp(max=total - 1)], 0).to(torch.int32).contiguous(), blocks


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + case["shape_seed"])
    s = {"case": case}
    hkv, d = case["hkv"], case["d"]
    if case["kind"] == "attend":
        new, ctx = lengths(case)
        s["tables"], blocks = tables(g, ctx)
        s["k"], s["v"], s["scales"] = pool(g, blocks, case)
        s["q"] = torch.randn((sum(new), case["hq"], d), generator=g, device=DEV, dtype=torch.bfloat16)
        s["indptr"] = torch.tensor(offsets(new), device=DEV, dtype=torch.int32)
        s["ctx"] = torch.tensor(ctx, device=DEV, dtype=torch.int32)
        s["max_new"], s["max_ctx"], s["scale"] = max(new), max(ctx), 1.0 / math.sqrt(d)
    elif case["kind"] == "write":
        t, hq = case["tokens"], case["hq"]
        blocks = t // BLOCK + t // (10 * BLOCK) + 4
        s["k"], s["v"], s["scales"] = pool(g, blocks, case)
        packed = torch.randn((t, hq + 2 * hkv, d), generator=g, device=DEV, dtype=torch.bfloat16) * 1.5
        s["q_in"], s["k_in"], s["v_in"] = packed.split((hq, hkv, hkv), dim=1)  # a fused projection's output
        s["slots"] = torch.randperm(blocks * BLOCK, generator=g, device=DEV)[:t].contiguous()
        s["pos"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV, dtype=torch.int32)
        half = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)
        s["wq"], s["wk"] = None, None
        if case["norm"]:
            s["wq"], s["wk"] = (1 + 0.2 * torch.randn((2, d), generator=g, device=DEV)).to(torch.bfloat16).unbind(0)
    else:
        lens = spans(case)
        s["tables"], blocks = tables(g, lens)
        s["k"], s["v"], s["scales"] = pool(g, blocks, case)
        s["indptr"] = torch.tensor(offsets(lens), device=DEV, dtype=torch.int32)
        s["rows"] = sum(lens)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return run_own(s)
    kind = s["case"]["kind"]
    return attend_plain(s) if kind == "attend" else write_plain(s) if kind == "write" else gather_plain(s)


def run_own(s):
    import paged_kv_cache_17_gb300 as pkv

    c = s["case"]
    if c["kind"] == "attend":
        lse = torch.empty(s["q"].shape[:2], device=DEV) if c["lse"] else None
        out = pkv.paged_prefill_attention(s["q"], s["indptr"], s["k"], s["v"], s["tables"], s["ctx"], s["scale"],
                                          causal=c["causal"], lse=lse, scales=s["scales"], max_context_len=s["max_ctx"])
        return (out, lse) if c["lse"] else out
    if c["kind"] == "write":
        q = pkv.qk_norm_rope_append(s["q_in"], s["k_in"], s["v_in"], s["pos"], s["slots"], s["k"], s["v"],
                                    q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, inv_freq=s["inv_freq"],
                                    interleaved=c["interleaved"], scales=s["scales"])
        return q, s["k"], s["v"]
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    k, v = (torch.empty((s["rows"], c["hkv"], c["d"]), device=DEV, dtype=dtype) for _ in range(2))
    pkv.paged_kv_gather(s["k"], s["v"], s["tables"], s["indptr"], k, v, scales=s["scales"])
    return k, v


def valued(x, scales, i):
    """Pool values in 32 bits."""
    return x.float() if scales is None else x.float() * scales[i][:, None]


def attend_plain(s):
    c = s["case"]
    b, hq, hkv, d, g = c["batch"], c["hq"], c["hkv"], c["d"], c["hq"] // c["hkv"]
    mq, mk = s["max_new"], s["max_ctx"]
    new = s["indptr"][1:] - s["indptr"][:-1]
    i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    real = i < new[:, None]
    row = (s["indptr"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(b, mq, hkv, g, d).permute(0, 2, 3, 1, 4).reshape(b, hkv, g * mq, d)
    pages = s["tables"][:, : (mk + BLOCK - 1) // BLOCK].long()
    k, v = (valued(x[pages], s["scales"], n).view(b, -1, hkv, d)[:, :mk].permute(0, 2, 1, 3)
            for n, x in enumerate((s["k"], s["v"])))
    sees = s["ctx"][:, None].expand(b, mq)
    if c["causal"]:
        sees = (s["ctx"] - new)[:, None] + i + 1
    hidden = (j >= sees[..., None])[:, None, None]
    score = torch.matmul(q, k.transpose(2, 3)).view(b, hkv, g, mq, mk).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
    most = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = score.sub_(most).exp_()
    total = p.sum(-1, keepdim=True)
    v = torch.where((j < s["ctx"][:, None])[:, None, :, None], v, 0)
    o = torch.matmul(p.view(b, hkv, g * mq, mk), v).view(b, hkv, g, mq, d) / total.clamp(min=1e-37)
    o = o.permute(0, 3, 1, 2, 4).reshape(b, mq, hq, d)
    out = torch.empty_like(s["q"])
    spare = torch.full((), s["q"].shape[0], device=DEV)
    at = torch.where(real, row, spare).view(-1)  # padded rows go behind the end
    out = torch.cat((out, out[:1])).index_copy_(0, at, o.reshape(-1, hq, d).to(out.dtype))[:-1]
    if not c["lse"]:
        return out
    lse = (most + total.log()).permute(0, 3, 1, 2, 4).reshape(-1, hq)
    return out, lse.new_empty((s["q"].shape[0] + 1, hq)).index_copy_(0, at, lse)[:-1]


def write_plain(s):
    c = s["case"]
    rot, half = c["rot"], c["rot"] // 2
    turn = s["pos"].double()[:, None] * s["inv_freq"]
    cos, sin = turn.cos().float()[:, None], turn.sin().float()[:, None]

    def turned(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        r = x[..., :rot]
        a, b = (r[..., ::2], r[..., 1::2]) if c["interleaved"] else (r[..., :half], r[..., half:])
        a, b = a * cos - b * sin, b * cos + a * sin
        r = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((r, x[..., rot:]), -1)

    def store(cache, x, i):
        flat = cache.view(-1, c["hkv"], c["d"])
        if s["scales"] is None:
            flat[s["slots"]] = x.to(cache.dtype)
        else:
            code = (x / s["scales"][i][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            flat.view(torch.uint8)[s["slots"]] = code.view(torch.uint8)

    store(s["k"], turned(s["k_in"], s["wk"]), 0)
    store(s["v"], s["v_in"].float(), 1)
    return turned(s["q_in"], s["wq"]).to(torch.bfloat16), s["k"], s["v"]


def gather_plain(s):
    c = s["case"]
    row = torch.arange(s["rows"], device=DEV)
    b = torch.searchsorted(s["indptr"][1:].long(), row, right=True)
    at = row - s["indptr"].long()[b]
    page = s["tables"].long()[b, at // BLOCK]
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    return tuple(valued(x[page, at % BLOCK], s["scales"], i).to(dtype) for i, x in enumerate((s["k"], s["v"])))


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    scales = s["scales"].double() if s["scales"] is not None else torch.ones((2, case["hkv"]), device=DEV, dtype=torch.float64)
    if case["kind"] == "attend":
        return exact_attend(case, s, scales)
    if case["kind"] == "write":
        return exact_write(case, s, scales)
    found = []
    for i, x in enumerate((s["k"], s["v"])):
        rows = [x[t.long()].double().flatten(0, 1)[:n] * scales[i][None, :, None] for t, n in zip(s["tables"], spans(case))]
        found.append(torch.cat(rows))
    return tuple(found)


def exact_attend(case, s, scales):
    new, ctx = lengths(case)
    if 4 * case["d"] * case["hq"] * sum(n * c for n, c in zip(new, ctx)) > 12e12:
        return None
    g, at = case["hq"] // case["hkv"], offsets(new)
    out = torch.zeros(s["q"].shape, device=DEV, dtype=torch.float64)
    lse = torch.full(s["q"].shape[:2], -math.inf, device=DEV, dtype=torch.float64)
    for b, (n, c) in enumerate(zip(new, ctx)):
        t = s["tables"][b, : (c + BLOCK - 1) // BLOCK].long()
        kv = [x[t].double().flatten(0, 1)[:c] * scales[i][None, :, None] for i, x in enumerate((s["k"], s["v"]))]
        for i0 in range(0, n, 512):
            i = torch.arange(i0, min(n, i0 + 512), device=DEV)
            far = c - n + i if case["causal"] else torch.full_like(i, c - 1)
            for h in range(case["hq"]):
                x = s["q"][at[b] + i, h].double() @ kv[0][:, h // g].T * s["scale"]
                x[torch.arange(c, device=DEV)[None, :] > far[:, None]] = -math.inf
                lse[at[b] + i, h] = torch.logsumexp(x, 1)
                out[at[b] + i, h] = torch.softmax(x, 1).nan_to_num(0) @ kv[1][:, h // g]
    return (out, lse) if case["lse"] else out


def exact_write(case, s, scales):
    """q rotated, and the pools with the chunk's rows in them (8-bit rows before rounding)."""
    half, done = case["rot"] // 2, []
    angle = (s["pos"].double()[:, None] * s["inv_freq"])[:, None, :]
    for x, w in ((s["q_in"], s["wq"]), (s["k_in"], s["wk"])):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
        y = x.clone()
        i = torch.arange(half, device=DEV)
        p, q = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
        z = torch.polar(torch.ones_like(angle), angle) * torch.complex(x[..., p], x[..., q])
        y[..., p], y[..., q] = z.real, z.imag
        done.append(y)
    pools = []
    for i, (cache, x) in enumerate(((s["k"], done[1]), (s["v"], s["v_in"].double()))):
        y = cache.double()
        x = x / scales[i][None, :, None]
        y.view(-1, case["hkv"], case["d"])[s["slots"]] = x.clamp(-448, 448) if case["e4m3"] else x
        pools.append(y)
    return done[0], pools[0], pools[1]
