"""The serving operators beside the composite delta, as cases to measure.

Three operators of one decode or prefill step of a multi-tenant batch:

* append: rotated keys and plain values written into a paged cache, queries rotated on the way;
* attend: attention over that cache for requests in groups, the requests of a group sharing a prefix
  whose keys and values are read once for all of them;
* sample: the next token of every row of logits by temperature, top-k, top-p and min-p from given uniforms.

``run`` computes them from elementary torch operations in 32 bits, or, with ``own`` set, through the
package's entry points.  A case's lengths follow from the case alone; a seed changes the values.
"""
import math

import numpy as np
import torch

own = False

BF16 = torch.bfloat16


# ------------------------------------------------------------------ cases
def listed():
    # 32 query and 8 key/value heads of 128 are the q (4096) and k/v (1024) projections of the benchmark's decode workloads.
    heads = dict(hq=32, hkv=8, d=128)
    return [
        # one decode token: latency alone
        dict(name="append-1", op="append", tokens=1, page=16, rot=128, interleaved=False, max_pos=8192, **heads),
        # the largest decode batch of the rank sweep, three padding tokens in it
        dict(name="append-256", op="append", tokens=256, page=16, rot=128, interleaved=False, max_pos=32768, **heads),
        # a prefill chunk as long as the sparse prefill batch
        dict(name="append-3250", op="append", tokens=3250, page=64, rot=128, interleaved=False, max_pos=8192, **heads),
        # one request behind a system prompt: latency alone
        dict(name="attend-1", op="attend", requests=1, groups=1, prefix=1000, suffix=37, queries=1, page=16, **heads),
        # the distinct decode batch's 32 requests behind one prompt, ragged answers so far
        dict(name="attend-32", op="attend", requests=32, groups=1, prefix=4099, suffix=384, queries=1, page=16, **heads),
        # a large decode batch behind a very long prompt: the products bound it
        dict(name="attend-256", op="attend", requests=256, groups=1, prefix=32768, suffix=512, queries=1, page=64, **heads),
        # tenants with a prompt each (ragged, one without any): the prefixes' bytes bound it
        dict(name="attend-tenants", op="attend", requests=64, groups=16, prefix=8192, suffix=700, queries=1, page=32, **heads),
        # drafted tokens to verify, a head of keys for each head of queries
        dict(name="attend-verify", op="attend", requests=24, groups=2, prefix=2048, suffix=1500, queries=8, page=64,
             hq=16, hkv=16, d=64),
        # prefill chunks of several requests behind their prompt
        dict(name="attend-chunk", op="attend", requests=6, groups=1, prefix=3001, suffix=1024, queries=1024, page=64, **heads),
        # one row of a large vocabulary: latency alone
        dict(name="sample-1", op="sample", rows=1, vocab=131072, dtype="float32", mixed=False),
        # the Zipf batch's 64 rows, a middling vocabulary, settings of their own per row
        dict(name="sample-64", op="sample", rows=64, vocab=32768, dtype="bfloat16", mixed=True),
        # the largest decode batch over an odd large vocabulary
        dict(name="sample-256", op="sample", rows=256, vocab=131001, dtype="bfloat16", mixed=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sample"])
    if op == "append":
        d = rng.choice([64, 128])
        return dict(op=op, tokens=_log(rng, 1, 4096), page=rng.choice([16, 32, 64, 128]),
                    rot=rng.choice([d, d, d // 2, 16]), interleaved=rng.random() < 0.4,
                    max_pos=_log(rng, 2048, 131072), hq=rng.choice([8, 16, 24, 32]), hkv=rng.choice([1, 2, 4, 8]), d=d)
    if op == "sample":
        return dict(op=op, rows=_log(rng, 1, 256), vocab=_log(rng, 1000, 131072),
                    dtype=rng.choice(["float32", "bfloat16"]), mixed=rng.random() < 0.8)
    hkv = rng.choice([1, 2, 4, 8])
    case = dict(op=op, requests=_log(rng, 1, 256), groups=1, prefix=_log(rng, 16, 32768), suffix=_log(rng, 1, 1500),
                queries=rng.choice([1, 1, 1, 1, rng.randint(2, 16), _log(rng, 17, 700)]),
                page=rng.choice([16, 32, 64, 128]), hq=hkv * rng.choice([1, 2, 4, 8]), hkv=hkv, d=rng.choice([64, 128]))
    if case["queries"] > 16:
        case["requests"] = min(case["requests"], 8)
    elif case["queries"] > 1:
        case["requests"] = min(case["requests"], 48)
    case["suffix"] = max(case["suffix"], case["queries"])
    case["groups"] = rng.randint(1, min(case["requests"], 16))
    most = work(listed()[5])["flops"]
    while work(case)["flops"] > most or case["groups"] * case["prefix"] > 131072:
        case["prefix"] = max(16, case["prefix"] // 2 + 1)
        case["suffix"] = max(case["queries"], case["suffix"] * 3 // 4)
    return case


def _lengths(case):
    """Query tokens, suffix lengths and group sizes of the requests, prefix lengths of the groups: of the case alone."""
    B, NG, Q = case["requests"], case["groups"], case["queries"]
    r = np.random.RandomState(17 * B + 31 * NG + 7 * Q + case["prefix"] + case["suffix"])
    q_len = np.full(B, 1) if Q == 1 else r.randint(1, Q + 1, B)
    q_len[r.randint(B)] = Q
    suffix = np.maximum(r.randint(1, case["suffix"] + 1, B), q_len)
    suffix[r.randint(B)] = case["suffix"]
    cuts = np.sort(r.choice(np.arange(1, B), NG - 1, replace=False)) if NG > 1 else np.zeros(0, int)
    group_offsets = np.concatenate([[0], cuts, [B]]).astype(np.int64)
    prefix = np.full(1, case["prefix"]) if NG == 1 else r.randint(case["prefix"] // 4, case["prefix"] + 1, NG)
    if NG > 2:
        prefix[r.randint(NG)] = 0
    return q_len, suffix, group_offsets, prefix


def work(case):
    if case["op"] == "append":
        T, rows = case["tokens"], 2 * case["hq"] + 4 * case["hkv"]
        return {"bytes": T * rows * case["d"] * 2 + T * case["rot"] * 4 + 8 * T,
                "flops": 3 * T * (case["hq"] + case["hkv"]) * case["rot"]}
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (4 if case["dtype"] == "float32" else 2) + 28 * case["rows"], "flops": 4 * n}
    q_len, suffix, go, prefix = _lengths(case)
    seen = 0
    for g in range(case["groups"]):
        seen += int(prefix[g]) * int(q_len[go[g]:go[g + 1]].sum())
    seen += int((q_len * suffix - q_len * (q_len - 1) // 2).sum())
    kv = int(prefix.sum() + suffix.sum()) * case["hkv"] * case["d"] * 4
    io = int(q_len.sum()) * case["hq"] * (case["d"] * 4 + 4)
    return {"bytes": kv + io, "flops": 4 * seen * case["hq"] * case["d"]}


# ------------------------------------------------------------------ inputs
def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def _prepare_append(case, seed, gen, r):
    T, hq, hkv, d, page = (case[k] for k in ("tokens", "hq", "hkv", "d", "page"))
    pages = max(8, 2 * (T // page + 1))
    s = dict(case)
    # q, k and v are slices of one projection's output, as a fused projection gives them
    qkv = _normal(gen, T, (hq + 2 * hkv) * d).to(BF16)
    s["q"] = qkv[:, :hq * d].view(T, hq, d)
    s["k"] = qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    s["v"] = qkv[:, (hq + hkv) * d:].view(T, hkv, d)
    slots = r.choice(pages * page, T, replace=False)
    if T >= 64:
        slots[r.choice(T, 3, replace=False)] = -1  # padding of a captured batch size
    s["slots"] = _dev(slots)
    s["positions"] = _dev(r.randint(0, case["max_pos"], T))
    half = case["rot"] // 2
    angle = np.arange(case["max_pos"])[:, None] * (10000.0 ** (-np.arange(half) / half))[None, :]
    s["rope"] = _dev(np.concatenate([np.cos(angle), np.sin(angle)], 1), torch.float32)
    # a page more than the cache has, for the plain form's padding tokens
    s["k_all"] = _normal(gen, pages + 1, hkv, page, d).to(BF16)
    s["v_all"] = _normal(gen, pages + 1, hkv, page, d).to(BF16)
    s["k_cache"], s["v_cache"] = s["k_all"][:pages], s["v_all"][:pages]
    s["q_out"] = torch.empty(T, hq, d, dtype=BF16, device="cuda")
    if own:
        import tenant_composite_lora_gb300 as tcl
        s["cache"] = tcl.LoraKvCache(pages, page, hkv, d, k=s["k_cache"], v=s["v_cache"])
    return s


def _prepare_attend(case, seed, gen, r):
    hq, hkv, d, page = (case[k] for k in ("hq", "hkv", "d", "page"))
    q_len, suffix, go, prefix = _lengths(case)
    B, NG, TQ = case["requests"], case["groups"], int(q_len.sum())
    sp, pp = -(-suffix // page), -(-prefix // page)
    total = int(sp.sum() + pp.sum())
    pages = total + 3
    order = r.permutation(pages)[:total]
    suffix_pages, prefix_pages = np.zeros((B, sp.max()), np.int64), np.zeros((NG, max(1, pp.max())), np.int64)
    at = 0
    for table, counts in ((prefix_pages, pp), (suffix_pages, sp)):
        for i, n in enumerate(counts):
            table[i, :n] = order[at:at + n]
            at += n
    s = dict(case)
    s["q"] = (1.5 * _normal(gen, TQ, hq, d)).to(BF16)
    s["k_cache"] = _normal(gen, pages, hkv, page, d).to(BF16)
    s["v_cache"] = _normal(gen, pages, hkv, page, d).to(BF16)
    q_off = np.concatenate([[0], np.cumsum(q_len)])
    s["q_offsets"], s["suffix_len"], s["suffix_pages"] = _dev(q_off), _dev(suffix), _dev(suffix_pages)
    s["group_offsets"], s["prefix_len"], s["prefix_pages"] = _dev(go), _dev(prefix), _dev(prefix_pages)
    s["scale"] = 1 / math.sqrt(d)
    s["out"] = torch.empty(TQ, hq, d, dtype=BF16, device="cuda")
    s["lse"] = torch.empty(TQ, hq, dtype=torch.float32, device="cuda")
    if own:
        import tenant_composite_lora_gb300 as tcl
        s["cache"] = tcl.LoraKvCache(pages, page, hkv, d, k=s["k_cache"], v=s["v_cache"])
        s["plan"] = tcl.LoraAttnPlan(B, NG, TQ, prefix_pages.shape[1], suffix_pages.shape[1], hq, hkv, d, page)
        s["plan"].build(s["q_offsets"], s["suffix_len"], s["suffix_pages"], TQ, pages,
                        s["group_offsets"], s["prefix_len"], s["prefix_pages"])
    else:  # where each padded place of the plain form lies
        Q, R = int(q_len.max()), int(np.diff(go).max())
        place = np.minimum(q_off[:-1, None] + np.arange(Q)[None, :], TQ - 1)
        member = np.minimum(go[:-1, None] + np.arange(R)[None, :], B - 1)
        group = np.searchsorted(go[1:], np.arange(B), side="right")
        s["place"], s["member"] = _dev(place, torch.int64), _dev(member, torch.int64)
        s["group"], s["within"] = _dev(group, torch.int64), _dev(np.arange(B) - go[:-1][group], torch.int64)
        s["q_len"] = _dev(q_len)
        b_of = np.repeat(np.arange(B), q_len)
        s["back"] = _dev(b_of * Q + np.arange(TQ) - q_off[b_of], torch.int64)
    return s


def _prepare_sample(case, seed, gen, r):
    T, V = case["rows"], case["vocab"]
    s = dict(case)
    # a broad body and a few likely tokens; some rows nearly flat, some masked by a grammar
    l = 2.5 * _normal(gen, T, V)
    likely = torch.randint(0, V, (T, 48), generator=gen, device="cuda")
    l.scatter_add_(1, likely, 4 + 9 * torch.rand(T, 48, generator=gen, device="cuda"))
    k = np.full(T, 50)
    p, tau, mp = np.full(T, 0.95), np.full(T, 0.8), np.zeros(T)
    if case["mixed"]:
        kind = r.randint(0, 16, T)
        l[_dev(kind == 1, torch.bool)] *= 0.2
        masked = _dev(kind == 2, torch.bool)[:, None] & (torch.rand(T, V, generator=gen, device="cuda") < 0.9)
        l.masked_fill_(masked, -math.inf)
        k = r.choice([0, 0, 20, 50, 200], T)
        p = r.choice([1.0, 0.8, 0.9, 0.95], T)
        mp = r.choice([0.0, 0.0, 0.02, 0.1], T)
        tau = np.where(kind >= 14, 0.0, r.uniform(0.5, 1.3, T))
    s["logits"] = l.to(getattr(torch, case["dtype"]))
    s["top_k"], s["top_p"] = _dev(k), _dev(p, torch.float32)
    s["temperature"], s["min_p"] = _dev(tau, torch.float32), _dev(mp, torch.float32)
    s["u"] = torch.rand(T, generator=gen, device="cuda")
    s["tokens"] = torch.empty(T, dtype=torch.int32, device="cuda")
    s["probs"] = torch.empty(T, dtype=torch.float32, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    r = np.random.RandomState(int(seed) % (1 << 31))
    return {"append": _prepare_append, "attend": _prepare_attend, "sample": _prepare_sample}[case["op"]](
        {k: v for k, v in case.items() if k != "name"}, seed, gen, r)


# ------------------------------------------------------------------ one pass
def run(s):
    if own:
        import tenant_composite_lora_gb300 as tcl
        if s["op"] == "append":
            tcl.kv_append(s["cache"], s["k"], s["v"], s["slots"], s["positions"], s["rope"], q=s["q"], q_out=s["q_out"],
                          interleaved=s["interleaved"])
            return s["q_out"], s["k_cache"], s["v_cache"]
        if s["op"] == "attend":
            tcl.prefix_attention(s["q"], s["cache"], s["plan"], s["scale"], out=s["out"], lse=s["lse"])
            return s["out"], s["lse"]
        tcl.sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], tokens=s["tokens"],
                   probs=s["probs"])
        return s["tokens"], s["probs"]
    return {"append": _append_plain, "attend": _attend_plain, "sample": _sample_plain}[s["op"]](s)


def _rotate(x, cos, sin, interleaved):
    """The first 2 * cos.shape[-1] elements of each head rotated; x float [T, H, D], cos and sin [T, 1, half]."""
    half = cos.shape[-1]
    rot, rest = x[..., :2 * half], x[..., 2 * half:]
    if interleaved:
        a, b = rot[..., 0::2], rot[..., 1::2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = rot[..., :half], rot[..., half:]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([rot, rest], -1)


def _append_plain(s):
    half = s["rot"] // 2
    row = s["rope"][s["positions"].long()][:, None, :]
    cos, sin = row[..., :half], row[..., half:]
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, s["interleaved"]))
    k = _rotate(s["k"].float(), cos, sin, s["interleaved"])
    slot = s["slots"].long()
    slot = torch.where(slot < 0, s["k_cache"].shape[0] * s["page"], slot)
    page, off = slot // s["page"], slot % s["page"]
    s["k_all"][page, :, off] = k.to(BF16)
    s["v_all"][page, :, off] = s["v"]
    return s["q_out"], s["k_cache"], s["v_cache"]


def _part(q, k, v, seen):
    """Attention of q [N, H, R, D] over k, v [N, H, L, D] where seen [N, 1, R or 1, L] is true: maxima, sums, products."""
    score = torch.matmul(q, k.transpose(-1, -2))
    score = torch.where(seen, score, -math.inf)
    m = score.amax(-1, keepdim=True)
    safe = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(score - safe)
    return m, e.sum(-1, keepdim=True), torch.matmul(e, v)


def _pages(cache, table):
    """[N, Hkv, L, D] in 32 bits of the pages that table [N, P] names."""
    x = cache[table.long()]
    N, P, H, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(N, H, P * page, D).float()


def _attend_plain(s):
    hkv, d = s["hkv"], s["d"]
    G = s["hq"] // hkv
    B, Q = s["place"].shape
    NG, R = s["member"].shape
    q = s["q"].float()[s["place"]] * s["scale"]
    q = q.view(B, Q, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, Q * G, d)
    # the requests' own keys: query i of n sees the first len - n + i + 1
    k, v = _pages(s["k_cache"], s["suffix_pages"]), _pages(s["v_cache"], s["suffix_pages"])
    at = torch.arange(k.shape[2], device="cuda")
    first = (s["suffix_len"] - s["q_len"])[:, None] + 1 + torch.arange(Q, device="cuda")[None, :]
    seen = at[None, None, :] < torch.minimum(first, s["suffix_len"][:, None])[:, :, None]
    own_part = _part(q, k, v, seen[:, :, None, :].expand(B, Q, G, -1).reshape(B, 1, Q * G, -1))
    # the groups' prefixes, for all requests of a group at once
    k, v = _pages(s["k_cache"], s["prefix_pages"]), _pages(s["v_cache"], s["prefix_pages"])
    at = torch.arange(k.shape[2], device="cuda")
    seen = (at[None, :] < s["prefix_len"][:, None])[:, None, None, :]
    qg = q[s["member"]].transpose(1, 2).reshape(NG, hkv, R * Q * G, d)
    shared = [x.view(NG, hkv, R, Q * G, -1).transpose(1, 2)[s["group"], s["within"]] for x in _part(qg, k, v, seen)]
    (m0, l0, o0), (m1, l1, o1) = own_part, shared
    m = torch.maximum(m0, m1)
    safe = torch.where(m == -math.inf, 0.0, m)
    w0, w1 = torch.exp(m0 - safe), torch.exp(m1 - safe)
    l = l0 * w0 + l1 * w1
    out = torch.where(l > 0, (o0 * w0 + o1 * w1) / torch.where(l > 0, l, 1.0), 0.0)
    lse = safe + torch.log(l)

    def rows(x):
        return x.view(B, hkv, Q, G, -1).permute(0, 2, 1, 3, 4).reshape(B * Q, hkv * G, -1)[s["back"]]

    return rows(out).to(BF16), rows(lse)[..., 0].contiguous()


def _sample_plain(s):
    l = s["logits"].float()
    V = l.shape[1]
    l = torch.where(torch.isnan(l), -math.inf, l)
    m = l.amax(-1, keepdim=True)
    greedy = s["temperature"] <= 0
    tau = torch.where(greedy, 1.0, s["temperature"])[:, None]
    e = torch.where(l == m, 1.0, torch.exp((l - m) * (1.0 / tau)))
    e = torch.where(l == -math.inf, 0.0, e)
    order = torch.sort(l, dim=-1, descending=True, stable=True).indices
    rank = torch.arange(V, device="cuda")[None, :]
    k = torch.where((s["top_k"] <= 0) | (s["top_k"] > V), V, s["top_k"])[:, None]
    k = torch.where(greedy[:, None], 1, k)
    es = torch.where(rank < k, e.gather(1, order), 0.0)
    mass = torch.cumsum(es, -1)
    before = torch.cat([torch.zeros_like(mass[:, :1]), mass[:, :-1]], -1)
    p = s["top_p"][:, None]
    keep = (before < p * mass[:, -1:]) | (p >= 1) | (rank == 0)
    keep = keep & (es >= s["min_p"].clamp(max=1)[:, None])
    kept = torch.zeros_like(e).scatter(1, order, torch.where(keep, es, 0.0))
    c = torch.cumsum(kept, -1)
    z = c[:, -1:]
    hit = (c > s["u"][:, None] * z) & (kept > 0)
    token = torch.where(hit, rank, V).amin(-1)
    last = torch.where(kept > 0, rank, -1).amax(-1)
    token = torch.where(token == V, last, token)
    prob = torch.where(token >= 0, kept.gather(1, token.clamp(min=0)[:, None])[:, 0] / z[:, 0], 0.0)
    return token.to(torch.int32), prob


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "attend": _attend_exact, "sample": _sample_exact}[case["op"]](s)


def _append_exact(s):
    half, page, hkv, d = s["rot"] // 2, s["page"], s["hkv"], s["d"]
    row = s["rope"].cpu().numpy().astype(np.float64)[s["positions"].cpu().numpy()]
    z = torch.from_numpy(row[:, :half] + 1j * row[:, half:]).cuda()[:, None, :]

    def turned(x):  # pairs as complex numbers, times cos + i sin
        x = x.double().clone()
        a, b = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if s["interleaved"] else (slice(0, half), slice(half, 2 * half))
        w = torch.complex(x[..., a].clone(), x[..., b].clone()) * z
        x[..., a], x[..., b] = w.real, w.imag
        return x

    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    k = turned(s["k"])
    slots = s["slots"].cpu().numpy()
    live = torch.from_numpy(np.flatnonzero(slots >= 0)).cuda()
    at = s["slots"].long()[live]
    k_cache[at // page, :, at % page] = k[live]
    v_cache[at // page, :, at % page] = s["v"].double()[live]
    return turned(s["q"]), k_cache, v_cache


def _attend_exact(s):
    hq, hkv, d, page = s["hq"], s["hkv"], s["d"], s["page"]
    G = hq // hkv
    q_off, suffix_len = s["q_offsets"].tolist(), s["suffix_len"].tolist()
    go, prefix_len = s["group_offsets"].tolist(), s["prefix_len"].tolist()
    out = torch.zeros(q_off[-1], hq, d, dtype=torch.float64, device="cuda")
    lse = torch.full((q_off[-1], hq), -math.inf, dtype=torch.float64, device="cuda")

    def keys(cache, table, n):
        x = cache[table[:-(-n // page)].long()].transpose(0, 1).reshape(hkv, -1, d)
        return x[:, :n].double()

    for g in range(s["groups"]):
        kp, vp = (keys(s[c], s["prefix_pages"][g], prefix_len[g]) for c in ("k_cache", "v_cache"))
        for b in range(go[g], go[g + 1]):
            n = q_off[b + 1] - q_off[b]
            k, v = (torch.cat([x, keys(s[c], s["suffix_pages"][b], suffix_len[b])], 1)
                    for x, c in ((kp, "k_cache"), (vp, "v_cache")))
            ends = prefix_len[g] + suffix_len[b] - n + 1 + torch.arange(n, device="cuda")
            for h in range(hkv):
                q = s["q"][q_off[b]:q_off[b + 1], h * G:(h + 1) * G].double()
                score = torch.einsum("ngd,kd->ngk", q, k[h]) * s["scale"]
                score.masked_fill_((torch.arange(k.shape[1], device="cuda")[None, :] >= ends[:, None])[:, None, :], -math.inf)
                out[q_off[b]:q_off[b + 1], h * G:(h + 1) * G] = torch.einsum("ngk,kd->ngd", torch.softmax(score, -1), v[h])
                lse[q_off[b]:q_off[b + 1], h * G:(h + 1) * G] = torch.logsumexp(score, -1)
    return out, lse


def _sample_exact(s):
    logits = s["logits"].double().cpu().numpy()
    T, V = logits.shape
    prob = np.zeros(T)
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, logits[t])
        order = np.argsort(-l, kind="stable")
        order = order[l[order] > -np.inf]
        if not order.size:
            continue
        tau, k = float(s["temperature"][t]), int(s["top_k"][t])
        p, mp, u = float(s["top_p"][t]), float(s["min_p"][t]), float(s["u"][t])
        if tau <= 0:
            prob[t] = 1.0
            continue
        order = order[:k] if 0 < k < V else order
        e = np.exp((l[order] - l[order[0]]) / tau)
        before = np.concatenate([[0.0], np.cumsum(e)[:-1]])
        keep = (e >= min(mp, 1.0)) & ((before < p * e.sum()) | (p >= 1) | (np.arange(e.size) == 0))
        order, e = order[keep], e[keep]
        by_index = np.argsort(order)
        c = np.cumsum(e[by_index])
        at = min(int(np.searchsorted(c, u * c[-1], side="right")), e.size - 1)
        prob[t] = e[by_index][at] / c[-1]
    return None, torch.from_numpy(prob)
