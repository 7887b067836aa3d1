"""The measured cases of differential attention over the paged cache: chunks of new tokens,
one token per sequence, and one token per sequence where sequences share a long prefix.

Heads come in pairs: output head p has the queries 2p and 2p + 1, reads the keys of kv heads 2n and
2n + 1 and, as one value twice as wide, the values of both; n is the pair of kv heads of p's group.
With A_m the softmax map of query 2p + m over keys 2n + m,

    out_p = out_scale * norm((A_0 - lam_p A_1) [V_2n, V_2n+1]),    norm(x) = x w / sqrt(mean(x^2) + eps).

Each case is run either through the package's public calls (`own` true) or in its plain form:
elementary torch operations in 32 bits, rounded once at the end.
"""
import math
import random

import torch

own = False

BLOCK = 16
D = 64  # elements of a head; a pair's value has 2 D
EPS = 1e-5
DEV = "cuda"


# ------------------------------------------------------------------ cases

def listed():
    return [
        # prompts of a batch of new requests, nothing cached yet, odd lengths
        chunk("chunk_prompts", 9, (257, 2048), (0, 0), 64, 16),
        # a chunk of a long document late in its prefill: the largest products
        chunk("chunk_long", 1, (4096, 4096), (28672, 28672), 64, 16),
        # speculated tokens of 24 running requests checked at once: few rows, long ragged contexts
        chunk("chunk_verify", 24, (3, 8), (1800, 12000), 64, 16, per_token=True),
        # chunks of four requests over an 8-bit cache, the widest query group
        chunk("chunk_e4m3", 4, (700, 1100), (3000, 9000), 128, 16, e4m3=True),
        # a decoder's tokens over an encoder's states kept in pages: no causal mask, no norm
        chunk("chunk_cross", 16, (1, 448), (750, 1500), 16, 4, causal=False, norm=False),
        # one user's next token over a short chat: nothing but latency
        decode("decode_one", 1, (777, 777), 64, 16),
        # one decode step of a batch of ordinary requests
        decode("decode_batch", 64, (512, 4096), 64, 16),
        # long contexts, the widest query group: the most bytes
        decode("decode_long", 8, (32768, 131072), 128, 16, per_token=True),
        # an 8-bit cache without shared heads
        decode("decode_e4m3", 33, (1000, 9001), 16, 16, e4m3=True, norm=False, fp32=True),
        # a batch of users of one system prompt, each with a conversation of its own
        shared("shared_prompt", 1, 256, 2048, (32, 512), 64, 16),
        # the samples of best-of-8 requests over an 8-bit cache
        shared("shared_fork_e4m3", 16, 8, 2000, (1, 256), 64, 16, e4m3=True),
        # two prompts and a few requests without one, a small group
        shared("shared_few", 2, 3, 784, (1, 90), 16, 8, alone=3),
    ]


def chunk(name, batch, new, past, hq, hkv, e4m3=False, causal=True, norm=True, per_token=False, shape_seed=1):
    return {"name": name, "kind": "chunk", "batch": batch, "new_min": new[0], "new_max": new[1], "past_min": past[0],
            "past_max": past[1], "hq": hq, "hkv": hkv, "e4m3": e4m3, "causal": causal, "norm": norm, "fp32": False,
            "per_token": per_token, "shape_seed": shape_seed}


def decode(name, batch, lens, hq, hkv, e4m3=False, norm=True, per_token=False, fp32=False, shape_seed=1):
    return {"name": name, "kind": "decode", "batch": batch, "len_min": lens[0], "len_max": lens[1], "hq": hq, "hkv": hkv,
            "e4m3": e4m3, "norm": norm, "per_token": per_token, "fp32": fp32, "shape_seed": shape_seed}


def shared(name, prompts, members, prefix, tails, hq, hkv, alone=0, e4m3=False, norm=True, per_token=False, fp32=False,
           shape_seed=1):
    return {"name": name, "kind": "shared", "prompts": prompts, "members": members, "alone": alone, "prefix": prefix,
            "len_min": tails[0], "len_max": tails[1], "hq": hq, "hkv": hkv, "e4m3": e4m3, "norm": norm,
            "per_token": per_token, "fp32": fp32, "shape_seed": shape_seed}


def spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    seed = rng.randrange(1 << 30)
    hq, hkv = rng.choice(((64, 16), (128, 16), (16, 4), (16, 16), (16, 8), (32, 8)))
    e4m3, norm, per_token = rng.random() < 0.4, rng.random() < 0.7, rng.random() < 0.4
    kind = rng.choice(("chunk", "decode", "shared"))
    if kind == "chunk":
        batch = spread(rng, 1, 24)
        past = spread(rng, 1, 16384) if rng.random() < 0.8 else 0
        room = (1 << 31) // (batch * hq)  # of score entries for a sequence, padded
        new = spread(rng, 1, 2048)
        while new > 1 and new * (past + new) > room:
            new = (new + 1) // 2
        causal = rng.random() < 0.8 or past < 2
        c = chunk("", batch, (rng.randint(1, new), new), (rng.randint(0 if causal else 1, past), past) if past else (0, 0),
                  hq, hkv, e4m3, causal, norm, per_token, seed)
    elif kind == "decode":
        batch = spread(rng, 1, 256)
        top = spread(rng, 1, min(131072, (1 << 19) // batch))
        c = decode("", batch, (rng.randint(0, top), top), hq, hkv, e4m3, norm, per_token, rng.random() < 0.3, seed)
    else:
        prompts, members = spread(rng, 1, 16), spread(rng, 1, 64)
        tail = spread(rng, 1, 1024)
        prefix = BLOCK * spread(rng, 1, min(512, max(1, (1 << 18) // (BLOCK * prompts * members))))
        c = shared("", prompts, members, prefix, (rng.randint(0, tail), tail), hq, hkv, rng.randint(0, 3), e4m3, norm,
                   per_token, rng.random() < 0.3, seed)
    del c["name"]
    return c


def lengths(case):
    """(new tokens, cached tokens seen) of every sequence: its own pages' tokens where a prefix is shared."""
    r = random.Random(case["shape_seed"])
    if case["kind"] == "chunk":
        new = [r.randint(case["new_min"], case["new_max"]) for _ in range(case["batch"])]
        past = [r.randint(case["past_min"], case["past_max"]) for _ in range(case["batch"])]
        return new, [p + n for n, p in zip(new, past)] if case["causal"] else past
    batch = case["batch"] if case["kind"] == "decode" else case["prompts"] * case["members"] + case["alone"]
    return [1] * batch, [r.randint(case["len_min"], case["len_max"]) for _ in range(batch)]


def offsets(lens):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return at


def work(case):
    hq, hkv, one = case["hq"], case["hkv"], 1 if case["e4m3"] else 2
    new, ctx = lengths(case)
    cached, seen = sum(ctx), list(ctx)
    if case["kind"] == "shared":
        cached += case["prompts"] * case["prefix"]
        seen = [n + (case["prefix"] if b < case["prompts"] * case["members"] else 0) for b, n in enumerate(ctx)]
    causal = case["kind"] == "chunk" and case["causal"]
    pairs = sum(n * c - (n * (n - 1) // 2 if causal else 0) for n, c in zip(new, seen))
    rows = sum(new)
    return {"bytes": rows * hq * D * (6 if case["fp32"] else 4) + cached * hkv * D * 2 * one
                     + hq * 2 * (rows if case["per_token"] else 1),
            "flops": (2 * D + 4 * D) * hq * pairs}


# ------------------------------------------------------------------ inputs

def pool(g, blocks, case):
    """A pool of random K and V (E4M3 codes with their scales, or bf16)."""
    shape = (blocks, BLOCK, case["hkv"], D)
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


def ints(values):
    return torch.tensor(values, device=DEV, dtype=torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + case["shape_seed"])
    new, ctx = lengths(case)
    s = {"case": case, "max_new": max(new), "max_ctx": max(ctx), "scale": 1.0 / math.sqrt(D)}
    if case["kind"] == "shared":
        prompts, members, prefix = case["prompts"], case["members"], case["prefix"]
        both, blocks = tables(g, [prefix] * prompts + ctx)
        s["prefix_tables"] = both[:prompts, : prefix // BLOCK].contiguous()
        s["tables"] = both[prompts:, : (max(ctx) + BLOCK - 1) // BLOCK or 1].contiguous()
        s["prefix_lens"] = ints([prefix] * prompts)
        # a prompt's members stand anywhere in the batch
        order = torch.randperm(len(ctx), generator=g, device=DEV).tolist()
        prefix_of = [-1] * len(ctx)
        for i, b in enumerate(order[: prompts * members]):
            prefix_of[b] = i // members
        # (lengths go with the sequence's place among the members: every seed has the same work)
        at = [0] * len(ctx)
        for i, b in enumerate(order):
            at[b] = i
        s["tables"], ctx = s["tables"][at].contiguous(), [ctx[i] for i in at]
        s["indptr"], s["seqs"] = ints(offsets([members] * prompts)), ints(order[: prompts * members])
        s["seq_prefix"] = ints(prefix_of)
    else:
        s["tables"], blocks = tables(g, ctx)
        s["indptr"] = ints(offsets(new))
    s["k"], s["v"], s["scales"] = pool(g, blocks, case)
    rows, heads = sum(new), case["hq"] // 2
    s["q"] = torch.randn((rows, case["hq"], D), generator=g, device=DEV, dtype=torch.bfloat16)
    s["ctx"] = ints(ctx)
    lam = (rows, heads) if case["per_token"] else (heads,)
    s["lam"] = 0.5 + 0.2 * torch.randn(lam, generator=g, device=DEV)
    s["w"] = (1 + 0.2 * torch.randn(2 * D, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
    s["out_scale"] = 0.45 if case["norm"] else 1.0
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    return run_own(s) if own else run_plain(s)


def run_own(s):
    import paged_kv_cache_17_gb300 as pkv

    c = s["case"]
    keys = dict(norm_weight=s["w"], eps=EPS, out_scale=s["out_scale"], scales=s["scales"], max_context_len=s["max_ctx"])
    if c["kind"] == "chunk":
        return pkv.paged_diff_prefill_attention(s["q"], s["indptr"], s["k"], s["v"], s["tables"], s["ctx"], s["scale"],
                                                s["lam"], causal=c["causal"], **keys)
    out = torch.empty((s["q"].shape[0], c["hq"] // 2, 2 * D), device=DEV,
                      dtype=torch.float32 if c["fp32"] else torch.bfloat16)
    if c["kind"] == "decode":
        return pkv.paged_diff_decode_attention(s["q"], s["k"], s["v"], s["tables"], s["ctx"], s["scale"], s["lam"], out,
                                               **keys)
    return pkv.cascade_diff_decode_attention(s["q"], s["k"], s["v"], s["prefix_tables"], s["prefix_lens"], s["indptr"],
                                             s["seqs"], s["seq_prefix"], s["tables"], s["ctx"], s["scale"], s["lam"],
                                             out, max_members=c["members"], max_prefix_len=c["prefix"], **keys)


def run_plain(s):
    c = s["case"]
    if c["kind"] == "chunk":
        new = s["indptr"][1:] - s["indptr"][:-1]
        return attend_plain(s, s["tables"], s["ctx"], s["max_ctx"], new, s["indptr"][:-1], s["max_new"], c["causal"])
    batch = s["q"].shape[0]
    first, ones = torch.arange(batch, device=DEV), torch.ones(batch, device=DEV, dtype=torch.long)
    if c["kind"] == "decode":
        return attend_plain(s, s["tables"], s["ctx"], s["max_ctx"], ones, first, 1, False)
    # every sequence's whole table: its prefix's blocks (whole ones), then its own
    with_prefix = (s["seq_prefix"] >= 0)[:, None]
    lead = torch.where(with_prefix, s["prefix_lens"][s["seq_prefix"].clamp(min=0).long()][:, None] // BLOCK, 0)
    wide = s["prefix_tables"].shape[1] + s["tables"].shape[1]
    j = torch.arange(wide, device=DEV)[None]
    front = s["prefix_tables"][s["seq_prefix"].clamp(min=0).long()]
    front = torch.cat((front, front.new_zeros((batch, s["tables"].shape[1]))), 1)
    back = torch.gather(s["tables"], 1, (j - lead).clamp(0, s["tables"].shape[1] - 1).long())
    whole = torch.where(j < lead, front, back)
    return attend_plain(s, whole, s["ctx"] + BLOCK * lead[:, 0], s["max_ctx"] + c["prefix"], ones, first, 1, False)


def valued(x, scales):
    """Pool values in 32 bits."""
    return x.float() if scales is None else x.float() * scales[:, None]


def attend_plain(s, table, ctx, mk, new, first, mq, causal):
    c = s["case"]
    b, hq, hkv = table.shape[0], c["hq"], c["hkv"]
    pairs, g, heads, mk = hkv // 2, hq // hkv, hq // 2, max(1, mk)
    i, j = torch.arange(mq, device=DEV), torch.arange(mk, device=DEV)
    real = i < new[:, None]
    row = (first[:, None] + i).clamp(max=s["q"].shape[0] - 1)
    pages = table[:, : (mk + BLOCK - 1) // BLOCK].long()
    sees = ctx[:, None].expand(b, mq)
    if causal:
        sees = (ctx - new)[:, None] + i + 1
    hidden = (j >= sees[..., None])[:, None, None]
    past = (j >= ctx[:, None])[:, None, :, None]
    o = torch.empty((b, mq, pairs, g, 2 * D), device=DEV)
    some = max(1, min(pairs, (1 << 32) // max(1, b * 2 * g * mq * mk)))  # pairs at a time
    for n in range(0, pairs, some):
        m = min(some, pairs - n)
        at = slice(2 * n, 2 * (n + m))
        k, v = (valued(x[:, :, at][pages], None if s["scales"] is None else s["scales"][t][at])
                .view(b, -1, m, 2, D)[:, :mk] for t, x in enumerate((s["k"], s["v"])))
        k, v = k.permute(0, 2, 3, 4, 1), v.permute(0, 2, 1, 3, 4).reshape(b, m, mk, 2 * D).masked_fill(past, 0)
        q = s["q"][:, 2 * n * g: 2 * (n + m) * g][row].float().view(b, mq, m, g, 2, D)
        both = []
        for t in range(2):
            x = torch.matmul(q[:, :, :, :, t].permute(0, 2, 3, 1, 4).reshape(b, m, g * mq, D), k[:, :, t])
            x = x.view(b, m, g, mq, mk).mul_(s["scale"]).masked_fill_(hidden, -math.inf)
            p = x.sub_(x.amax(-1, keepdim=True).clamp(min=-1e30)).exp_()
            total = p.sum(-1, keepdim=True)
            both.append(torch.matmul(p.view(b, m, g * mq, mk), v).view(b, m, g, mq, 2 * D) / total.clamp(min=1e-37))
        lam = s["lam"][..., n * g: (n + m) * g]
        lam = lam[row].view(b, mq, m, g).permute(0, 2, 3, 1)[..., None] if c["per_token"] else lam.view(m, g, 1, 1)
        o[:, :, n: n + m] = (both[0] - lam * both[1]).permute(0, 3, 1, 2, 4)
    if s["w"] is not None:
        o = o * torch.rsqrt((o * o).mean(-1, keepdim=True) + EPS) * s["w"].float()
    o = (o * s["out_scale"]).view(b * mq, heads, 2 * D)
    dtype = torch.float32 if c["fp32"] else torch.bfloat16
    spare = s["q"].shape[0]  # padded rows go behind the end
    out = torch.empty((spare + 1, heads, 2 * D), device=DEV, dtype=dtype)
    return out.index_copy_(0, torch.where(real, row, spare).view(-1), o.to(dtype))[:-1]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    """Sequence by sequence and head by head from the definition."""
    if work(case)["flops"] > 12e12:
        return None
    s = prepare(case, seed)
    hq, g = case["hq"], case["hq"] // case["hkv"]
    causal = case["kind"] == "chunk" and case["causal"]
    ctx, rows = s["ctx"].tolist(), s["q"].shape[0]
    starts = s["indptr"].tolist() if case["kind"] == "chunk" else list(range(rows + 1))
    scales = s["scales"].double() if s["scales"] is not None else torch.ones((2, case["hkv"]), device=DEV, dtype=torch.float64)
    out = torch.zeros((rows, hq // 2, 2 * D), device=DEV, dtype=torch.float64)
    prefix_of = s["seq_prefix"].tolist() if case["kind"] == "shared" else [-1] * len(ctx)
    for b, own_len in enumerate(ctx):
        ids, c, n = s["tables"][b, : (own_len + BLOCK - 1) // BLOCK], own_len, starts[b + 1] - starts[b]
        if prefix_of[b] >= 0:
            ids, c = torch.cat((s["prefix_tables"][prefix_of[b]], ids)), c + case["prefix"]
        if n == 0 or c == 0:
            continue
        k, v = (x[ids.long()].double().flatten(0, 1)[:c] * scales[t][None, :, None] for t, x in enumerate((s["k"], s["v"])))
        value = v.reshape(c, case["hkv"] // 2, 2 * D)
        for i0 in range(0, n, 512):
            i = torch.arange(i0, min(n, i0 + 512), device=DEV)
            far = c - n + i if causal else torch.full_like(i, c - 1)
            mask = torch.arange(c, device=DEV)[None, :] > far[:, None]
            for kh in range(0, case["hkv"], 2):
                for p in range(kh // 2 * g, (kh // 2 + 1) * g):
                    a = []
                    for t in range(2):
                        x = s["q"][starts[b] + i, 2 * p + t].double() @ k[:, kh + t].T * s["scale"]
                        a.append(torch.softmax(x.masked_fill(mask, -math.inf), 1).nan_to_num(0) @ value[:, kh // 2])
                    lam = (s["lam"][starts[b] + i, p][:, None] if case["per_token"] else s["lam"][p]).double()
                    out[starts[b] + i, p] = a[0] - lam * a[1]
    if s["w"] is not None:
        out = out / (out.pow(2).mean(-1, keepdim=True) + EPS).sqrt() * s["w"].double()
    return out * s["out_scale"]
