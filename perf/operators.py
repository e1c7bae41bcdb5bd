"""The operators of the paged KV cache: their cases, their plain forms and what they cost.

Two operators.  `append` writes new tokens' keys and values into a paged cache, rotating keys (and the
same tokens' queries) by position on the way; the pages hold bf16, or e4m3 codes with a power-of-two scale
for each block of 16 tokens and KV head.  `attend` is softmax attention over the positions that a
selection lists, read through the page table from either kind of page.

With `own` false, run() computes them with elementary torch operations in 32 bits (rotation angles in 64);
with `own` true it calls the package.  Sizes are those of the framework's workloads (128k, 1m, 10m, decode)
and smaller and odder ones around them.
"""
import math

import numpy as np
import torch

own = False

SCALE_BLOCK = 16        # tokens that share a scale
MIN_EXP = -64           # smallest scale 2^-64
E4M3_MAX = 448.0


def listed():
    return [
        # The decode workload's step: 8 sequences of 1M tokens, a token each.
        dict(name="append_token_8x1m", op="append", fmt="e4m3", B=8, Nq=1, Hq=32, Hkv=4, d=128, page=64,
             pos=1 << 20, rot=128, inter=False, ragged=False, fused=True),
        # A larger odd batch at 128k in bf16 pages, half of each head rotated, pairs side by side.
        dict(name="append_token_61_bf16", op="append", fmt="bf16", B=61, Nq=1, Hq=16, Hkv=2, d=128, page=16,
             pos=131072, rot=64, inter=True, ragged=False, fused=False),
        # A padded batch of prompts of unequal lengths, an empty one among them; small heads.
        dict(name="append_ragged_7", op="append", fmt="e4m3", B=7, Nq=1021, Hq=24, Hkv=8, d=64, page=32,
             pos=5000, rot=64, inter=False, ragged=True, fused=False),
        # The 128k workload's chunk for two sequences, bf16 pages, sliced from one projection.
        dict(name="append_chunk_bf16", op="append", fmt="bf16", B=2, Nq=4096, Hq=16, Hkv=2, d=128, page=128,
             pos=126976, rot=128, inter=False, ragged=False, fused=True),
        # The last 32k chunk of a 10M context.
        dict(name="append_chunk_32k", op="append", fmt="e4m3", B=1, Nq=32768, Hq=32, Hkv=4, d=128, page=64,
             pos=10452992, rot=128, inter=False, ragged=False, fused=True),
        # One sequence of 10M tokens, one new query: latency, and offsets past 32 bits.
        dict(name="attend_token_10m", op="attend", fmt="e4m3", B=1, Nq=1, T=10485760, Hq=32, Hkv=4, d=128,
             page=64, R=4096, W=512, S=4, ragged=False),
        # The decode workload's step: 8 sequences of 1M tokens.
        dict(name="attend_token_8x1m", op="attend", fmt="e4m3", B=8, Nq=1, T=1 << 20, Hq=32, Hkv=4, d=128,
             page=64, R=4096, W=512, S=4, ragged=False),
        # A serving batch at 128k, bf16 pages.
        dict(name="attend_token_64_bf16", op="attend", fmt="bf16", B=64, Nq=1, T=131072, Hq=16, Hkv=2, d=128,
             page=128, R=4096, W=512, S=4, ragged=False),
        # An odd batch with rows of unequal length, empty ones among them; 3 query heads to a KV head.
        dict(name="attend_ragged_33", op="attend", fmt="e4m3", B=33, Nq=1, T=8192, Hq=24, Hkv=8, d=64, page=16,
             R=512, W=64, S=4, ragged=True),
        # A few queries of a 128k prompt's end, an odd number, bf16 pages.
        dict(name="attend_chunk_251_bf16", op="attend", fmt="bf16", B=1, Nq=251, T=131072, Hq=16, Hkv=2, d=128,
             page=64, R=4096, W=512, S=4, ragged=False),
        # A chunk of the 1m workload (2048 long-range keys), 8-bit pages.
        dict(name="attend_chunk_1k", op="attend", fmt="e4m3", B=1, Nq=1024, T=1 << 20, Hq=32, Hkv=4, d=128,
             page=64, R=2048, W=512, S=4, ragged=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    c = dict(fmt=rng.choice(["e4m3", "bf16", "e4m3"]), d=rng.choice([64, 128]), Hkv=rng.choice([1, 2, 3, 4, 8]),
             page=rng.choice([16, 32, 64, 128, 256]))
    c["Hq"] = c["Hkv"] * rng.choice([1, 2, 3, 4, 6, 8])
    if rng.random() < 0.5:
        B = _log_int(rng, 1, 64)
        Nq = rng.choice([1, _log_int(rng, 1, max(1, 32768 * 24 * 128 // (B * c["Hq"] * c["d"])))])
        rot = rng.choice([c["d"], c["d"] // 2, 32])
        return dict(c, op="append", B=B, Nq=min(Nq, 32768 // B), pos=_log_int(rng, 1, 10000000), rot=rot,
                    inter=rng.random() < 0.3, ragged=rng.random() < 0.4, fused=rng.random() < 0.5)
    R, W, S = _log_int(rng, 16, 4096) // 4 * 4, _log_int(rng, 3, 512), rng.choice([0, 1, 4])
    B = rng.choice([1, 1, _log_int(rng, 1, 64)])
    row = (R + W + S) * c["Hkv"] * c["d"]
    Nq = rng.choice([1, _log_int(rng, 1, max(1, min(1024, 1024 * 2564 * 512 // (2 * B * row))))])
    T = max(8192, _log_int(rng, 8192, max(8192, (1 << 31) // (B * c["Hkv"] * c["d"]))) // 4096 * 4096)
    return dict(c, op="attend", B=B, Nq=Nq, T=T, R=R, W=W, S=S, ragged=rng.random() < 0.4)


# ---- sizes that do not depend on the seed -----------------------------------------------------------------

def _n_new(c):
    """New tokens of each sequence of an append."""
    B, Nq = c["B"], c["Nq"]
    if not c["ragged"] or B == 1:
        return [Nq] * B
    return [Nq * ((b + B // 2) % B) // (B - 1) for b in range(B)]


def _counts(c):
    """Listed keys of each query row of an attend."""
    rows, s = c["B"] * c["Nq"], c["R"] + c["W"] + c["S"]
    if not c["ragged"] or rows == 1:
        return np.full(rows, s, np.int64)
    return s * ((np.arange(rows, dtype=np.int64) + rows // 2) % rows) // (rows - 1)


def work(case):
    c = case
    elt, hkv, hq, d = (1 if c["fmt"] == "e4m3" else 2), c["Hkv"], c["Hq"], c["d"]
    if c["op"] == "append":
        n = sum(_n_new(c))
        scales = n * 2 * hkv * 4 / SCALE_BLOCK if c["fmt"] == "e4m3" else 0
        return {"bytes": n * (2 * hkv * d * (2 + elt) + 2 * hq * d * 2) + scales + 8 * c["B"],
                "flops": n * (hkv + hq) * c["rot"] * 3}
    counts = _counts(c)
    total = int(counts.sum())
    # keys read by several queries count once: their expected number among the long-range buckets
    keys = total
    if c["Nq"] > 1 and not c["ragged"]:
        share = c["R"] / max(1, c["T"] - c["W"] - c["Nq"] - c["S"])
        far = (c["T"] - c["W"] - c["Nq"]) * (1 - (1 - min(1.0, share)) ** c["Nq"])
        keys = min(total, int(c["B"] * (far + c["W"] + c["Nq"] + c["S"])))
    row = 2 * hkv * d * elt + (2 * hkv * 4 / SCALE_BLOCK if c["fmt"] == "e4m3" else 0)
    return {"bytes": keys * row + total * 4 + len(counts) * (hq * (2 * d * 2 + 4) + 4),
            "flops": 4 * total * hq * d}


# ---- inputs -----------------------------------------------------------------------------------------------

def _pool(g, fmt, n_pages, page, hkv, d, unit):
    """Pages of values of about `unit` each, and the scales of 8-bit ones' blocks."""
    x = torch.randn(n_pages, page, hkv, d, dtype=torch.bfloat16, device="cuda", generator=g)
    if fmt == "bf16":
        return x.mul_(unit), None
    x = x.mul_(96).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    e = torch.randint(-1, 2, (n_pages, page // SCALE_BLOCK, hkv), device="cuda", generator=g)
    return x, torch.exp2((e + math.floor(math.log2(unit / 96))).float())


def _cache(g, c, n_pages):
    K, ks = _pool(g, c["fmt"], n_pages, c["page"], c["Hkv"], c["d"], 1 / math.sqrt(c["d"]))
    V, vs = _pool(g, c["fmt"], n_pages, c["page"], c["Hkv"], c["d"], 1.0)
    return K, V, None if ks is None else torch.stack([ks, vs], 2).contiguous()


def _handle(s):
    """The cache object that a program keeps."""
    if own:
        import long_context_indexing_b200 as lsa
        s["lsa"] = lsa
        s["cache"] = lsa.LsaPagedKV(s["K"], s["V"], s["table"], s["scales"])
    return s


def _prepare_append(c, g):
    B, Nq, Hq, Hkv, d, page = (c[k] for k in ("B", "Nq", "Hq", "Hkv", "d", "page"))
    start = c["pos"] + torch.randint(0, 64, (B,), device="cuda", generator=g)
    # only the pages that the call touches are in the pool: it reads no others
    span = (Nq + page - 2) // page + 1
    n_pages = B * span + 3
    table = torch.full((B, (c["pos"] + 64 + Nq) // page + 2), -1, dtype=torch.int64, device="cuda")
    perm = torch.randperm(n_pages, device="cuda", generator=g)[:B * span].view(B, span)
    table.scatter_(1, start[:, None] // page + torch.arange(span, device="cuda"), perm)
    K, V, scales = _cache(g, c, n_pages)
    qkv = torch.randn(B, Nq, Hq + 2 * Hkv, d, device="cuda", generator=g)
    # norms differ from token to token, as a projection gives them
    qkv.mul_(torch.exp2(torch.rand(B, Nq, 1, 1, device="cuda", generator=g) * 4 - 3))
    q, k, v = qkv.to(torch.bfloat16).split([Hq, Hkv, Hkv], 2)
    if not c["fused"]:
        q, k, v = q.contiguous(), k.contiguous(), v.contiguous()
    r = c["rot"]
    inv = (1e6 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)).float()
    return dict(case=c, K=K, V=V, scales=scales, table=table.to(torch.int32), start=start.to(torch.int32),
                n_new=torch.tensor(_n_new(c), dtype=torch.int32, device="cuda") if c["ragged"] else None,
                q=q, k=k, v=v, q_out=torch.zeros(B, Nq, Hq, d, dtype=torch.bfloat16, device="cuda"), inv_freq=inv)


def _select(c, g):
    """Selections as the bucket retrieval makes them: sinks, whole buckets of 4-key groups spread over a block of
    4096 keys, the recent window; a row's count cuts it short."""
    B, Nq, T, R, W, S = (c[k] for k in ("B", "Nq", "T", "R", "W", "S"))
    nb, blocks = -(-R // 256), max(1, (T - W - Nq) // 4096)
    m = torch.rand(B * Nq, blocks * 16, device="cuda", generator=g).topk(min(nb, blocks * 16), 1).indices
    j = torch.arange(64, device="cuda")
    group = (m // 16)[..., None] * 1024 + j * 16 + (j * 7 + (m % 16)[..., None] + m[..., None] // 16) % 16
    far = (group[..., None] * 4 + torch.arange(4, device="cuda")).reshape(B * Nq, -1)[:, :R]
    pos = (T - Nq + torch.arange(Nq, device="cuda")).repeat(B)[:, None]
    rows = [torch.arange(S, device="cuda").expand(B * Nq, S), far, pos - W + 1 + torch.arange(W, device="cuda")]
    idx = torch.cat(rows, 1)
    idx = torch.nn.functional.pad(idx, (0, R + W + S - idx.shape[1]), value=-1)
    counts = torch.from_numpy(_counts(c)).cuda().clamp_(max=sum(x.shape[1] for x in rows))
    idx = idx.masked_fill(torch.arange(idx.shape[1], device="cuda") >= counts[:, None], -1)
    return idx.view(B, Nq, -1).to(torch.int32), counts.view(B, Nq).to(torch.int32)


def _prepare_attend(c, g):
    B, Nq, T, Hq, Hkv, d, page = (c[k] for k in ("B", "Nq", "T", "Hq", "Hkv", "d", "page"))
    n_pages = B * (T // page)
    table = torch.randperm(n_pages, device="cuda", generator=g).view(B, T // page)
    K, V, scales = _cache(g, c, n_pages)
    idx, counts = _select(c, g)
    # each query points at one of its keys, as far as a matching key's logit of about 8 wants it
    at = (torch.rand(B, Nq, device="cuda", generator=g) * counts).long().clamp_(max=idx.shape[2] - 1)
    t = idx.gather(2, at[..., None])[..., 0].long().clamp_(min=0)
    slot = table.gather(1, t // page) * page + t % page
    one = K.view(torch.uint8 if scales is not None else K.dtype).view(-1, Hkv, d)[slot]
    one = (one.view(K.dtype) if scales is not None else one).float()
    one = one / one.norm(dim=-1, keepdim=True).clamp_(min=1e-6)
    q = 8 * (one[:, :, :, None] * math.sqrt(d)
             + 0.3 * torch.randn(B, Nq, Hkv, Hq // Hkv, d, device="cuda", generator=g))
    return dict(case=c, K=K, V=V, scales=scales, table=table.to(torch.int32), indices=idx, counts=counts,
                Q=q.view(B, Nq, Hq, d).to(torch.bfloat16))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return _handle((_prepare_append if case["op"] == "append" else _prepare_attend)(case, g))


# ---- one pass ---------------------------------------------------------------------------------------------

def run(state):
    s = state
    if s["case"]["op"] == "append":
        if own:
            s["lsa"].lsa_paged_append(s["cache"], s["k"], s["v"], s["start"], n_new=s["n_new"], q=s["q"],
                                      q_out=s["q_out"], inv_freq=s["inv_freq"], interleaved=s["case"]["inter"])
        else:
            _append(s)
        return dict(K=s["K"], V=s["V"], scales=s["scales"], q=s["q_out"])
    if own:
        o, lse = s["lsa"].lsa_paged_attn(s["cache"], s["Q"], s["indices"], s["counts"], return_lse=True)
    else:
        o, lse = _attend(s)
    return dict(o=o, lse=lse)


def _rotate(x, cos, sin, inter):
    """Rotation of the first 2 * cos.shape[-1] values of each head."""
    x, r = x.float(), 2 * cos.shape[-1]
    a, b = (x[..., :r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    y = (a * cos - b * sin, b * cos + a * sin)
    return torch.cat([torch.stack(y, -1).flatten(-2) if inter else torch.cat(y, -1), x[..., r:]], -1)


def _append(s):
    c, B, Nq = s["case"], s["case"]["B"], s["case"]["Nq"]
    t = s["start"].long()[:, None] + torch.arange(Nq, device="cuda")
    angle = t[..., None, None].double() * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    k, q = _rotate(s["k"], cos, sin, c["inter"]), _rotate(s["q"], cos, sin, c["inter"])
    n_new = s["n_new"].long() if s["n_new"] is not None else torch.full((B,), Nq, device="cuda")
    live = torch.arange(Nq, device="cuda") < n_new[:, None]
    s["q_out"].copy_(torch.where(live[..., None, None], q.to(torch.bfloat16), s["q_out"]))
    slot = (s["table"].long().gather(1, t // c["page"]) * c["page"] + t % c["page"])[live]
    k, v = k[live], s["v"].float()[live]
    if s["scales"] is None:
        s["K"].view(-1, c["Hkv"], c["d"])[slot] = k.to(torch.bfloat16)
        s["V"].view(-1, c["Hkv"], c["d"])[slot] = v.to(torch.bfloat16)
        return
    first = s["start"].long()
    page = s["table"].long().gather(1, first[:, None] // c["page"])[:, 0]
    head = (page * c["page"] + first % c["page"]) // SCALE_BLOCK      # the block of each sequence's first new token
    kept = torch.where(n_new > 0, first % SCALE_BLOCK, 0)             # its tokens from before the call
    _store(s["K"], s["scales"], 0, k, slot, head, kept)
    _store(s["V"], s["scales"], 1, v, slot, head, kept)


def _codes(x):
    return x.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _store(pool, scales, which, x, slot, head, kept):
    hkv, d = pool.shape[2:]
    flat, old = pool.view(torch.uint8).view(-1, hkv, d), scales.view(-1, 2, hkv)[:, which]
    block = slot // SCALE_BLOCK
    amax = torch.zeros_like(old).scatter_reduce(0, block[:, None].expand(-1, hkv), x.abs().amax(-1), "amax")
    m, e = torch.frexp(amax)                                          # amax <= 448 * 2^k: 448 = 0.875 * 2^9
    new = torch.exp2((e - 9 + (m > 0.875)).clamp(min=MIN_EXP).float())
    h, n = head[kept > 0], kept[kept > 0]
    new[h] = torch.maximum(new[h], old[h])
    # tokens that were in the block before take the new scale
    at = h[:, None] * SCALE_BLOCK + torch.arange(SCALE_BLOCK, device="cuda")
    before = flat[at].view(torch.float8_e4m3fn).float() * (old[h] / new[h])[:, None, :, None]
    stays = (torch.arange(SCALE_BLOCK, device="cuda") >= n[:, None])[..., None, None]
    flat[at] = torch.where(stays, flat[at], _codes(before).view(torch.uint8))
    flat[slot] = _codes(x / new[block][..., None]).view(torch.uint8)
    old[block] = new[block]


def _gather(s, pool, which, slot):
    hkv, d = pool.shape[2:]
    if s["scales"] is None:
        return pool.view(-1, hkv, d)[slot].float()
    x = pool.view(torch.uint8).view(-1, hkv, d)[slot].view(torch.float8_e4m3fn).float()
    return x.mul_(s["scales"].view(-1, 2, hkv)[:, which][slot // SCALE_BLOCK][..., None])


def _attend(s):
    c, idx = s["case"], s["indices"].long()
    B, Nq, n = idx.shape
    dead = (torch.arange(n, device="cuda") >= s["counts"][..., None])[:, :, None, None]
    t = idx.clamp(min=0)
    slot = s["table"].long()[torch.arange(B, device="cuda")[:, None, None], t // c["page"]] * c["page"] + t % c["page"]
    q = s["Q"].float().view(B, Nq, c["Hkv"], -1, c["d"])
    z = q @ _gather(s, s["K"], 0, slot).permute(0, 1, 3, 4, 2) / math.sqrt(c["d"])
    z = z.masked_fill(dead, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    p = (z - m).exp()
    total = p.sum(-1, keepdim=True)
    o = p @ _gather(s, s["V"], 1, slot).transpose(2, 3) / total.clamp(min=1e-30)
    return o.view(B, Nq, c["Hq"], c["d"]).to(torch.bfloat16), (m + total.log()).view(B, Nq, c["Hq"])


# ---- the definition in 64 bits ----------------------------------------------------------------------------

def exact(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if case["op"] == "append":
        return _exact_append(_prepare_append(case, g))
    return _exact_attend(_prepare_attend(case, g))


def _grid(x):
    """x on the e4m3 grid: 4 significant bits, the spacing never below 2^-9, halves to even, at most 448."""
    _, e = torch.frexp(x)
    step = torch.exp2((e - 4).clamp(min=-9).double())
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_append(s):
    c, r = s["case"], s["case"]["rot"]
    page, n_new = c["page"], _n_new(c)
    K, V, q_out = s["K"].double(), s["V"].double(), s["q_out"].double()
    scales = None if s["scales"] is None else s["scales"].double()
    freq = s["inv_freq"].double()
    for b in range(c["B"]):
        n, t0 = n_new[b], int(s["start"][b])
        if n == 0:
            continue
        t = torch.arange(t0, t0 + n, device="cuda")
        turn = torch.polar(torch.ones(n, r // 2, dtype=torch.float64, device="cuda"), t.double()[:, None] * freq)
        rows = s["table"][b].long()[t // page] * page + t % page
        turned = []
        for x in (s["q"][b, :n].double(), s["k"][b, :n].double()):
            if c["inter"]:
                z = torch.view_as_complex(x[..., :r].reshape(n, -1, r // 2, 2).contiguous()) * turn[:, None]
                y = torch.view_as_real(z).flatten(-2)
            else:
                z = torch.complex(x[..., :r // 2], x[..., r // 2:r]) * turn[:, None]
                y = torch.cat([z.real, z.imag], -1)
            turned.append(torch.cat([y, x[..., r:]], -1))
        q_out[b, :n] = turned[0]
        for which, pool, x in ((0, K, turned[1]), (1, V, s["v"][b, :n].double())):
            flat = pool.view(-1, c["Hkv"], c["d"])
            if scales is None:
                flat[rows] = x
                continue
            # the sequence's touched blocks, first to last, each padded to 16 tokens
            lead = t0 % SCALE_BLOCK
            nb = (lead + n + SCALE_BLOCK - 1) // SCALE_BLOCK
            wide = torch.zeros(nb * SCALE_BLOCK, c["Hkv"], c["d"], dtype=torch.float64, device="cuda")
            wide[lead:lead + n] = x
            amax = wide.view(nb, SCALE_BLOCK, c["Hkv"], c["d"]).abs().amax((1, 3))
            sc = torch.exp2(torch.ceil(torch.log2(amax / E4M3_MAX)).clamp(min=MIN_EXP))
            # a logarithm next to a whole number may have gone to its other side
            sc = torch.where((amax <= E4M3_MAX * (sc / 2)) & (sc > 2.0 ** MIN_EXP), sc / 2, sc)
            sc = torch.where(amax > E4M3_MAX * sc, sc * 2, sc)
            pick = [0] + [SCALE_BLOCK * i - lead for i in range(1, nb)]
            blk = rows[torch.tensor(pick, device="cuda")] // SCALE_BLOCK
            stored = scales.view(-1, 2, c["Hkv"])
            if lead:
                was = stored[blk[0], which]
                sc[0] = torch.maximum(sc[0], was)
                early = blk[0] * SCALE_BLOCK + torch.arange(lead, device="cuda")
                flat[early] = _grid(flat[early] * (was / sc[0])[None, :, None])
            flat[rows] = _grid(x / sc[torch.arange(lead, lead + n, device="cuda") // SCALE_BLOCK][..., None])
            stored[blk, which] = sc
    return dict(K=K, V=V, scales=scales, q=q_out)


def _exact_attend(s):
    c = s["case"]
    B, Nq, Hkv, d, page = (c[k] for k in ("B", "Nq", "Hkv", "d", "page"))
    o = torch.zeros(B, Nq, c["Hq"], d, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Nq, c["Hq"]), -math.inf, dtype=torch.float64, device="cuda")
    counts = s["counts"].tolist()

    def values(pool, which, rows):
        if s["scales"] is None:
            return pool.view(-1, Hkv, d)[rows].double()
        x = pool.view(torch.uint8).view(-1, Hkv, d)[rows].view(torch.float8_e4m3fn).double()
        return x * s["scales"].view(-1, 2, Hkv)[rows // SCALE_BLOCK, which].double()[..., None]

    for b in range(B):
        for i in range(Nq):
            n = counts[b][i]
            if n == 0:
                continue
            t = s["indices"][b, i, :n].long()
            rows = s["table"][b].long()[t // page] * page + t % page
            z = torch.einsum("ghd,tgd->ght", s["Q"][b, i].double().view(Hkv, -1, d), values(s["K"], 0, rows))
            z = z / math.sqrt(d)
            lse[b, i] = torch.logsumexp(z, -1).flatten()
            o[b, i] = torch.einsum("ght,tgd->ghd", torch.softmax(z, -1), values(s["V"], 1, rows)).reshape(-1, d)
    return dict(o=o, lse=lse)
