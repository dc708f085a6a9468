"""Cases of the attention-layer operators, to time them and to compare their outputs.

A model that mixes Gated DeltaNet-2 layers with softmax-attention layers runs
three more operators in each attention layer: the per-head RMS norm of queries
and keys with the rotary position embedding, the same on the way into a paged
key/value cache, and the attention of a chunk of new tokens over that cache.

``run`` computes them with elementary torch operations in fp32 (``own`` false)
or through this package (``own`` true); ``exact`` computes them in fp64.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
EPS = 1e-6


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one token of one sequence: the launch and its latency, nothing else
        dict(name="norm_rope_token", op="norm_rope", dtype="bf16", T=1, HQ=16, HK=16, D=128, rot=128,
             interleaved=False, scaling="none", packed=False, max_pos=4096),
        # a decode step of 128 sequences at long positions, context extended 8 times by parts
        dict(name="norm_rope_decode", op="norm_rope", dtype="bf16", T=128, HQ=32, HK=8, D=128, rot=128,
             interleaved=False, scaling="parts", packed=True, max_pos=131072),
        # a long prefill: half of each head rotated, q and k views of one packed projection
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", T=32768, HQ=32, HK=32, D=128, rot=64,
             interleaved=False, scaling="none", packed=True, max_pos=32768),
        # odd counts, interleaved pairs, small heads, fp16, positions divided by a factor
        dict(name="norm_rope_odd", op="norm_rope", dtype="fp16", T=4099, HQ=15, HK=5, D=64, rot=64,
             interleaved=True, scaling="linear", packed=False, max_pos=16384),
        # a decode step: one token of each of 128 sequences joins the cache
        dict(name="append_decode", op="append", dtype="bf16", N=128, new_lo=1, new_hi=1, past_lo=1, past_hi=8191,
             HQ=32, HKV=8, D=128, rot=128, interleaved=False, scaling="none", norm=True, page=64, layout="nhd",
             lens_seed=1),
        # a packed prefill of ragged prompts, 32768 tokens or so, small pages
        dict(name="append_varlen", op="append", dtype="bf16", N=8, new_lo=64, new_hi=8192, past_lo=0, past_hi=0,
             HQ=32, HKV=32, D=128, rot=64, interleaved=False, scaling="none", norm=True, page=16, layout="nhd",
             lens_seed=2),
        # continued chunks, head-major pages of an odd size, fp16, interleaved, no norm, an empty sequence
        dict(name="append_odd", op="append", dtype="fp16", N=9, new_lo=0, new_hi=1000, past_lo=0, past_hi=3001,
             HQ=12, HKV=4, D=64, rot=32, interleaved=True, scaling="parts", norm=False, page=40, layout="hnd",
             lens_seed=3),
        # one new token of one short sequence: latency
        dict(name="attn_token", op="attn", dtype="bf16", N=1, new_lo=1, new_hi=1, past_lo=776, past_hi=776, HQ=16,
             HKV=4, D=128, page=64, layout="nhd", causal=True, window=-1, lens_seed=4),
        # a decode step of 128 sequences of ragged lengths up to 8192 keys
        dict(name="attn_decode", op="attn", dtype="bf16", N=128, new_lo=1, new_hi=1, past_lo=1, past_hi=8191, HQ=32,
             HKV=8, D=128, page=64, layout="nhd", causal=True, window=-1, lens_seed=5),
        # a chunk of a long prompt: 2048 new tokens after 30720 cached ones
        dict(name="attn_chunk", op="attn", dtype="bf16", N=1, new_lo=2048, new_hi=2048, past_lo=30720,
             past_hi=30720, HQ=32, HKV=8, D=128, page=64, layout="nhd", causal=True, window=-1, lens_seed=6),
        # a batch of ragged chunks, one head group per query head, some with cached prefixes, small pages
        dict(name="attn_varlen", op="attn", dtype="bf16", N=8, new_lo=1, new_hi=4096, past_lo=0, past_hi=4096, HQ=16,
             HKV=16, D=128, page=16, layout="hnd", causal=True, window=-1, lens_seed=7),
        # small heads in groups of three, fp16, a sliding window, an odd page size, an empty sequence
        dict(name="attn_odd", op="attn", dtype="fp16", N=7, new_lo=0, new_hi=700, past_lo=0, past_hi=3000, HQ=12,
             HKV=4, D=64, page=48, layout="nhd", causal=True, window=500, lens_seed=8),
    ]


def log_int(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    while True:
        c = dict(op=rng.choice(["norm_rope", "append", "attn"]), dtype=rng.choice(["bf16", "bf16", "fp16"]),
                 D=rng.choice([64, 128, 128]))
        group = rng.choice([1, 1, 2, 3, 4, 5, 8, 16])
        kv = rng.choice([1, 2, 3, 4, 8, 16, 32])
        if group * kv > 40:
            continue
        rotary = dict(rot=rng.choice([r for r in (16, 32, 64, 96, 128) if r <= c["D"]]),
                      interleaved=rng.random() < 0.4, scaling=rng.choice(["none", "linear", "parts"]))
        if c["op"] == "norm_rope":
            c.update(T=log_int(rng, 1, 32768), HQ=group * kv, HK=kv, **rotary, packed=rng.random() < 0.5,
                     max_pos=log_int(rng, 4096, 131072))
            if c["T"] * (c["HQ"] + c["HK"]) * c["D"] > 32768 * 64 * 128:
                continue
            return c
        n = log_int(rng, 1, 128)
        new = 1 if rng.random() < 0.35 else log_int(rng, 2, 8192)
        past = log_int(rng, 1, 32768)
        c.update(N=n, new_lo=rng.choice([0, 1, new]) if n > 1 else new, new_hi=new, past_lo=rng.choice([0, 1, past]),
                 past_hi=past, HQ=group * kv, HKV=kv, page=rng.choice([16, 32, 48, 64, 64, 128, 256]),
                 layout=rng.choice(["nhd", "nhd", "hnd"]), lens_seed=rng.randrange(1 << 20))
        length = c["past_hi"] + c["new_hi"]
        if c["op"] == "append":
            c.update(**rotary, norm=rng.random() < 0.6)
            if n * new * (c["HQ"] + 2 * kv) * c["D"] > 32768 * 96 * 128 or n * length * kv * c["D"] > 1 << 30:
                continue
        else:
            c.update(causal=rng.random() < 0.85, window=-1)
            if c["causal"] and rng.random() < 0.3:
                c["window"] = log_int(rng, 16, 4096)
            if n * c["HQ"] * new * length > 1 << 31 or n * length * kv * c["D"] > 1 << 30:
                continue
        if sum(lengths(c)[0]) == 0:
            continue
        return c


def lengths(c):
    """(new tokens, cached tokens before them) of each sequence of a case."""
    rng = random.Random(c["lens_seed"])
    new = [rng.randint(c["new_lo"], c["new_hi"]) for _ in range(c["N"])]
    past = [rng.randint(c["past_lo"], c["past_hi"]) for _ in range(c["N"])]
    return new, past


def keys_seen(c):
    """Number of (new token, key) pairs that the case's mask leaves."""
    total = 0
    for n, p in zip(*lengths(c)):
        if not c["causal"]:
            total += n * (n + p)
        elif c["window"] < 0:
            total += n * p + n * (n + 1) // 2
        else:
            total += sum(min(p + i + 1, c["window"] + 1) for i in range(n))
    return total


def keys_needed(c):
    """Number of cached tokens that some new token of the case attends to."""
    total = 0
    for n, p in zip(*lengths(c)):
        if n:
            total += n + p if not c["causal"] or c["window"] < 0 else n + min(p, c["window"])
    return total


def work(c):
    if c["op"] == "norm_rope":
        elements = c["T"] * (c["HQ"] + c["HK"]) * c["D"]
        return {"bytes": 4 * elements + 4 * c["T"] + 4 * c["D"] + 4 * c["rot"], "flops": 8 * elements}
    new, past = lengths(c)
    tokens = sum(new)
    if c["op"] == "append":
        pages = sum(-(-(n + p) // c["page"]) - p // c["page"] for n, p in zip(new, past) if n)
        elements = tokens * (c["HQ"] + 2 * c["HKV"]) * c["D"]
        return {"bytes": 4 * elements + 4 * pages + 8 * c["N"], "flops": 8 * elements}
    keys = keys_needed(c)
    byte = 2 * 2 * tokens * c["HQ"] * c["D"] + 4 * tokens * c["HQ"]
    byte += 2 * 2 * keys * c["HKV"] * c["D"] + 4 * -(-keys // c["page"]) + 8 * c["N"]
    return {"bytes": byte, "flops": 4 * keys_seen(c) * c["HQ"] * c["D"]}


# ------------------------------------------------------------------ inputs
def frequencies(c):
    """Angle per position of each rotated pair (fp64), and the factor on cos and sin."""
    i = torch.arange(0, c["rot"], 2, dtype=torch.float64, device="cuda")
    f = 10000.0 ** (-i / c["rot"])
    if c["scaling"] == "linear":
        return f / 4.0, 1.0
    if c["scaling"] == "parts":
        # pairs that turn less than once in the trained context are slowed by
        # the factor, those that turn over 32 times are left, a ramp between
        factor, trained = 8.0, 16384
        ramp = ((trained * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
        return f * ramp + f / factor * (1.0 - ramp), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def paged(c, gen, dtype):
    """A paged cache with stale contents, and the page table of the case's sequences in random page order."""
    new, past = lengths(c)
    total = [n + p for n, p in zip(new, past)]
    counts = [-(-t // c["page"]) for t in total]
    spare = 3
    pages, width = sum(counts) + spare, max(1, max(counts))
    shape = (pages, c["page"], c["HKV"], c["D"])
    order = torch.randperm(pages, device="cuda", generator=gen).to(torch.int32)
    col = torch.arange(width, device="cuda")
    count = torch.tensor(counts, device="cuda")
    first = count.cumsum(0) - count
    table = order[(first[:, None] + col).clamp(max=pages - 1)]
    table = torch.where(col < count[:, None], table, torch.zeros_like(table)).contiguous()
    if c["layout"] == "hnd":
        shape = (pages, c["HKV"], c["page"], c["D"])
    caches = torch.randn((2,) + shape, device="cuda", dtype=dtype, generator=gen)
    if c["layout"] == "hnd":
        caches = caches.transpose(2, 3)
    ints = dict(device="cuda", dtype=torch.int32)
    cu = torch.tensor([0] + new, **ints).cumsum(0, dtype=torch.int32)
    return dict(k_cache=caches[0], v_cache=caches[1], table=table, cu=cu, kv_lens=torch.tensor(total, **ints),
                tokens=sum(new), widest=max(new), longest=max(total))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    c = case
    dtype = DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(shape, device="cuda", dtype=dtype, generator=gen)

    s = dict(c)
    if c["op"] != "attn":
        s["freq"], s["factor"] = frequencies(c)
        s["q_weight"] = 1.0 + 0.1 * normal(c["D"])
        s["k_weight"] = 1.0 + 0.1 * normal(c["D"])
    if c["op"] == "norm_rope":
        s["pos"] = torch.randint(0, c["max_pos"], (c["T"],), device="cuda", dtype=torch.int32, generator=gen)
        if c["packed"]:
            x = normal(c["T"], c["HQ"] + 2 * c["HK"], c["D"])  # queries, keys and values of one projection
            s["q"], s["k"] = x[:, :c["HQ"]], x[:, c["HQ"]:c["HQ"] + c["HK"]]
        else:
            s["q"], s["k"] = normal(c["T"], c["HQ"], c["D"]), normal(c["T"], c["HK"], c["D"])
        return s
    s.update(paged(c, gen, dtype))
    s["q"] = normal(s["tokens"], c["HQ"], c["D"])
    if c["op"] == "append":
        s["k"], s["v"] = normal(s["tokens"], c["HKV"], c["D"]), normal(s["tokens"], c["HKV"], c["D"])
    return s


# --------------------------------------------------------------- the passes
def run(state):
    if own:
        return run_own(state)
    return {"norm_rope": plain_norm_rope, "append": plain_append, "attn": plain_attn}[state["op"]](state)


def run_own(s):
    from gated_deltanet_prefill_gb300 import attn
    if s["op"] == "attn":
        return attn.paged_attn_fwd(s["q"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu"],
                                   causal=s["causal"], window_left=s["window"], return_lse=True)
    rotary = dict(inv_freq=s["freq"], rope_factor=s["factor"], interleaved=s["interleaved"], eps=EPS)
    if s["op"] == "norm_rope":
        return attn.qk_norm_rope(s["q"], s["k"], s["pos"], norm=True, q_weight=s["q_weight"],
                                 k_weight=s["k_weight"], **rotary)
    weights = dict(q_weight=s["q_weight"], k_weight=s["k_weight"]) if s["norm"] else {}
    q_out = attn.append_kv(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["kv_lens"], s["cu"], q=s["q"],
                           norm=s["norm"], **weights, **rotary)
    return q_out, s["k_cache"], s["v_cache"]


def plain_norm(x, weight):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()


def plain_rotate(x, pos, s):
    """x [T, H, D] in fp32, its first rot channels rotated by the tokens' positions."""
    rot = s["rot"]
    angle = pos.float()[:, None, None] * s["freq"].float()
    cos, sin = angle.cos() * s["factor"], angle.sin() * s["factor"]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def plain_norm_rope(s):
    q = plain_rotate(plain_norm(s["q"].float(), s["q_weight"]), s["pos"], s)
    k = plain_rotate(plain_norm(s["k"].float(), s["k_weight"]), s["pos"], s)
    return q.to(s["q"].dtype), k.to(s["k"].dtype)


def token_places(s):
    """Sequence and place in the cached sequence of each new token."""
    t = torch.arange(s["tokens"], device="cuda")
    seq = torch.searchsorted(s["cu"][1:].long(), t, right=True)
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    return seq, t - s["cu"].long()[seq] + s["kv_lens"].long()[seq] - new[seq]


def plain_append(s):
    seq, pos = token_places(s)
    q, k = s["q"].float(), s["k"].float()
    if s["norm"]:
        q, k = plain_norm(q, s["q_weight"]), plain_norm(k, s["k_weight"])
    q, k = plain_rotate(q, pos, s), plain_rotate(k, pos, s)
    page = s["table"][seq, pos // s["page"]].long()
    slot = pos % s["page"]
    s["k_cache"][page, slot] = k.to(s["k"].dtype)
    s["v_cache"][page, slot] = s["v"]
    return q.to(s["q"].dtype), s["k_cache"], s["v_cache"]


def plain_attn(s):
    n, hq, hkv, d = s["N"], s["HQ"], s["HKV"], s["D"]
    wide, long = s["widest"], s["longest"]
    cu, total = s["cu"].long(), s["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    row, col = torch.arange(wide, device="cuda"), torch.arange(long, device="cuda")
    # padded queries [N, HKV, rows, D] and keys and values [N, HKV, keys, D]
    at = (cu[:-1, None] + row).clamp(max=s["tokens"] - 1)
    q = s["q"][at].float().view(n, wide, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(n, hkv, -1, d)
    page = s["table"][:, col // s["page"]].long()
    k = s["k_cache"][page, col % s["page"]].float().permute(0, 2, 1, 3)
    v = s["v_cache"][page, col % s["page"]].float().permute(0, 2, 1, 3)
    scores = (q @ k.transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, hkv, wide, hq // hkv, long)
    pos = (total - new)[:, None] + row
    seen = (col < total[:, None])[:, None, :].expand(n, wide, long)
    if s["causal"]:
        seen = seen & (col <= pos[..., None])
        if s["window"] >= 0:
            seen = seen & (col >= pos[..., None] - s["window"])
    scores.masked_fill_(~seen[:, None, :, None, :], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = scores.sub_(top).exp_()
    norm = p.sum(-1)
    lse = norm.log() + top[..., 0]
    o = (p.view(n, hkv, -1, long) @ v).view(n, hkv, wide, hq // hkv, d)
    o = torch.where(norm[..., None] > 0, o / norm[..., None], torch.zeros_like(o))
    # back to the packed tokens
    seq, place = token_places(s)
    i = place - (total - new)[seq]
    return o[seq, :, i].reshape(-1, hq, d).to(s["q"].dtype), lse[seq, :, i].reshape(-1, hq)


# -------------------------------------------------------------- the definition
def exact_rotated(x, pos, weight, s):
    """Norm (with a weight) and rotation of x [T, H, D] in fp64, pairs as complex numbers."""
    x = x.double()
    if weight is not None:
        x = x / (x.square().sum(-1, keepdim=True) / s["D"] + EPS).sqrt() * weight.double()
    turn = torch.polar(torch.full_like(s["freq"], s["factor"]) * torch.ones(len(pos), 1, device="cuda"),
                       torch.outer(pos.double(), s["freq"]))[:, None]
    rot = s["rot"]
    if s["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:2], rot // 2, 2).contiguous()) * turn
        y = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        y = torch.cat([z.real, z.imag], -1)
    return torch.cat([y, x[..., rot:]], -1)


def exact_attn(s):
    """Sequence by sequence and head by head, from gathered keys and values."""
    hq, hkv, d = s["HQ"], s["HKV"], s["D"]
    out = torch.zeros(s["tokens"], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((s["tokens"], hq), -math.inf, dtype=torch.float64, device="cuda")
    start = 0
    for i, (new, past) in enumerate(zip(*lengths(s))):
        if not new:
            continue
        pages = s["table"][i, :-(-(new + past) // s["page"])].long()
        ks = s["k_cache"][pages].flatten(0, 1)[:new + past]
        vs = s["v_cache"][pages].flatten(0, 1)[:new + past]
        col = torch.arange(new + past, device="cuda")
        for a in range(0, new, 2048):
            b = min(new, a + 2048)
            pos = torch.arange(past + a, past + b, device="cuda")[:, None]
            hidden = torch.zeros(b - a, new + past, dtype=torch.bool, device="cuda")
            if s["causal"]:
                hidden |= col > pos
                if s["window"] >= 0:
                    hidden |= col < pos - s["window"]
            for h in range(hq):
                g = h // (hq // hkv)
                x = s["q"][start + a:start + b, h].double() @ ks[:, g].double().T / math.sqrt(d)
                x = x.masked_fill(hidden, -math.inf)
                z = torch.logsumexp(x, -1)
                out[start + a:start + b, h] = torch.exp(x - z[:, None]) @ vs[:, g].double()
                lse[start + a:start + b, h] = z
        start += new
    return out, lse


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attn":
        # fp64 runs at about 1 TFLOP/s here
        dense = sum(n * (n + p) for n, p in zip(*lengths(case))) * 4.0 * case["HQ"] * case["D"]
        return exact_attn(s) if dense < 6e12 else None
    if case["op"] == "norm_rope":
        return exact_rotated(s["q"], s["pos"], s["q_weight"], s), exact_rotated(s["k"], s["pos"], s["k_weight"], s)
    weights = (s["q_weight"], s["k_weight"]) if s["norm"] else (None, None)
    seq, pos = [], []
    for i, (new, past) in enumerate(zip(*lengths(case))):
        seq += [i] * new
        pos += range(past, past + new)
    seq, pos = torch.tensor(seq, device="cuda"), torch.tensor(pos, device="cuda")
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    at = s["table"][seq, pos // s["page"]].long(), pos % s["page"]
    k_cache[at] = exact_rotated(s["k"], pos, weights[1], s)
    v_cache[at] = s["v"].double()
    return exact_rotated(s["q"], pos, weights[0], s), k_cache, v_cache
