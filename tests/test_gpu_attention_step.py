"""The paged append and the attention over shared prefixes against their
formulas in 64 bits.

Tolerances, from the roundings of the formulas (u = 2^-8, the unit roundoff
of bf16):
 * a rotated element: one rounding to bf16, after fp32 products of its pair:
   u |ref| + 2^-21 (|a| + |b|);
 * an attention output: its own rounding, u |out|; the rounding of each weight
   to bf16, u sum p |v|; the scores' fp32 error e (at most head_dim products,
   2^-17 scale sum |q k|), which scales each weight by at most 1 + 2 e both in
   the numerator and the sum; 2^-14 sum p |v| for exp and the fp32 sums;
 * lse: e + 2^-20 (1 + |lse|).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def built():
    from tenant_composite_lora_gb300 import build
    build.build()


def dev(a, dtype=torch.int32):
    return torch.as_tensor(np.ascontiguousarray(a)).to("cuda", dtype)


def rand(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)


def gen_of(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ------------------------------------------------------------------ append
def rope_table(max_pos, rot):
    half = rot // 2
    ang = np.arange(max_pos)[:, None] * (10000.0 ** (-np.arange(half) / max(half, 1)))[None, :]
    return dev(np.concatenate([np.cos(ang), np.sin(ang)], 1), torch.float32)


def rotated(x, rope, pos, interleaved):
    """(reference in 64 bits, |a| + |b| of each element's pair)."""
    x = x.double()
    rot = rope.shape[1]
    half = rot // 2
    c, s = rope.double()[pos.long()][:, None, :half], rope.double()[pos.long()][:, None, half:]
    ia = torch.arange(0, rot, 2, device="cuda") if interleaved else torch.arange(half, device="cuda")
    ib = ia + 1 if interleaved else ia + half
    a, b = x[..., ia], x[..., ib]
    ref, mag = x.clone(), torch.zeros_like(x)
    ref[..., ia], ref[..., ib] = a * c - b * s, b * c + a * s
    mag[..., ia] = a.abs() + b.abs()
    mag[..., ib] = a.abs() + b.abs()
    return ref, mag


@pytest.mark.parametrize("T", [1, 2, 37, 300])
@pytest.mark.parametrize("d,rot,page,hq,hkv", [(128, 128, 16, 32, 8), (128, 64, 64, 5, 1), (64, 64, 32, 8, 8),
                                               (64, 16, 128, 6, 3), (128, 0, 16, 4, 2)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_matches_the_formula(T, d, rot, page, hq, hkv, interleaved):
    import tenant_composite_lora_gb300 as tcl
    g, r = gen_of(T + d + rot), np.random.RandomState(T)
    pages, max_pos = T // page + 3, 5000
    qkv = rand(g, T, (hq + 2 * hkv) * d + 24)  # a fused projection's output with room to spare
    q, k = qkv[:, :hq * d].view(T, hq, d), qkv[:, hq * d:(hq + hkv) * d].view(T, hkv, d)
    v = qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d].view(T, hkv, d)
    slots = r.choice(pages * page, T, replace=False)
    if T > 2:
        slots[1] = -1
    pos = dev(r.randint(0, max_pos, T))
    rope = rope_table(max_pos, rot) if rot else None
    cache = tcl.LoraKvCache(pages, page, hkv, d, k=rand(g, pages, hkv, page, d), v=rand(g, pages, hkv, page, d))
    k0, v0 = cache.k.clone(), cache.v.clone()
    q_out = torch.full((T, hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tcl.kv_append(cache, k, v, dev(slots), pos if rot else None, rope, q=q, q_out=q_out, interleaved=interleaved,
                  status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    live = np.flatnonzero(slots >= 0)
    at = torch.from_numpy(slots[live]).cuda()
    if rot:
        rq, mq = rotated(q, rope, pos, interleaved)
        rk, mk = rotated(k, rope, pos, interleaved)
    else:
        rq, rk = q.double(), k.double()
        mq, mk = torch.zeros_like(rq), torch.zeros_like(rk)
    assert bool(((q_out.double() - rq).abs() <= U * rq.abs() + 2.0 ** -21 * mq).all())
    got_k, got_v = cache.k[at // page, :, at % page].double(), cache.v[at // page, :, at % page]
    assert bool(((got_k - rk[live]).abs() <= U * rk[live].abs() + 2.0 ** -21 * mk[live]).all())
    assert torch.equal(got_v, v[live])
    # nothing else changed
    cache.k[at // page, :, at % page] = k0[at // page, :, at % page]
    cache.v[at // page, :, at % page] = v0[at // page, :, at % page]
    assert torch.equal(cache.k, k0) and torch.equal(cache.v, v0)


def test_append_without_queries_and_in_place():
    import tenant_composite_lora_gb300 as tcl
    g = gen_of(3)
    T, hq, hkv, d, page = 9, 4, 2, 64, 16
    k, v, q = rand(g, T, hkv, d), rand(g, T, hkv, d), rand(g, T, hq, d)
    pos, rope, slots = dev(np.arange(T) * 31), rope_table(512, d), dev(np.arange(T) + 5)
    a, b = tcl.LoraKvCache(2, page, hkv, d), tcl.LoraKvCache(2, page, hkv, d)
    tcl.kv_append(a, k, v, slots, pos, rope)
    out = torch.empty_like(q)
    tcl.kv_append(b, k, v, slots, pos, rope, q=q, q_out=out)
    tcl.kv_append(b, k, v, slots, pos, rope, q=q)  # in place
    torch.cuda.synchronize()
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(out, q)
    tcl.kv_append(a, k[:0], v[:0], slots[:0], pos[:0], rope)  # no tokens: nothing to do


def test_append_leaves_bad_tokens_out():
    import tenant_composite_lora_gb300 as tcl
    n = tcl.native
    g = gen_of(4)
    T, hq, hkv, d, page = 4, 2, 1, 64, 16
    k, v, q = rand(g, T, hkv, d), rand(g, T, hkv, d), rand(g, T, hq, d)
    rope = rope_table(8, d)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = tcl.LoraKvCache(2, page, hkv, d)
    out = torch.zeros_like(q)
    for slots, pos, bit, k_rows, q_rows in (([0, 32, 2, 3], [0, 1, 2, 3], n.LORA_DEV_BAD_SLOT, [0, 2, 3], 4),
                                            ([0, -2, 2, 3], [0, 1, 2, 3], n.LORA_DEV_BAD_SLOT, [0, 2, 3], 4),
                                            ([0, 1, 2, 3], [0, 1, 8, -1], n.LORA_DEV_BAD_POSITION, [0, 1], 2)):
        status.zero_()
        cache.k.zero_()
        out.zero_()
        tcl.kv_append(cache, k, v, dev(slots), dev(pos), rope, q=q, q_out=out, status=status)
        torch.cuda.synchronize()
        assert int(status) == bit
        assert sorted(np.flatnonzero(cache.k[:, 0].float().abs().sum(-1).flatten().cpu().numpy()).tolist()) == k_rows
        assert int((out.float().abs().sum((1, 2)) > 0).sum()) == q_rows


def test_append_refuses_what_it_cannot_take():
    import tenant_composite_lora_gb300 as tcl
    g = gen_of(5)
    T, hkv, d = 3, 2, 64
    cache = tcl.LoraKvCache(1, 16, hkv, d)
    k, slots, pos = rand(g, T, hkv, d), dev([0, 1, 2]), dev([0, 1, 2])
    with pytest.raises(ValueError, match="k: shape"):
        tcl.kv_append(cache, k[:, :1], k, slots)
    with pytest.raises(ValueError, match="v: bf16"):
        tcl.kv_append(cache, k, k.float(), slots)
    with pytest.raises(ValueError, match="heads must be contiguous"):
        tcl.kv_append(cache, k.transpose(1, 2).contiguous().transpose(1, 2), k, slots)
    with pytest.raises(ValueError, match="positions holds 2"):
        tcl.kv_append(cache, k, k, slots, pos[:2], rope_table(8, d))
    for rot in (8, 80):  # not a multiple of 16; above head_dim
        with pytest.raises(tcl.LoraError):
            tcl.kv_append(cache, k, k, slots, pos, torch.zeros(8, rot, device="cuda"))
    odd = torch.zeros(T, hkv * d + 4, dtype=torch.bfloat16, device="cuda")[:, :hkv * d].view(T, hkv, d)
    with pytest.raises(tcl.LoraError):  # a token stride that is no multiple of 8 elements
        tcl.kv_append(cache, odd, k, slots)
    for args in ((0, 16, 2, 64), (2, 24, 2, 64), (2, 16, 2, 96), (2, 16, 257, 64)):
        t = torch.zeros(max(1, math.prod(args)), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(tcl.LoraError):
            tcl.lora_kv_cache_create(*args, t, t)


# ------------------------------------------------------------------ attention
class Batch:
    """A batch in a scattered paged cache whose unused places hold NaN."""

    def __init__(self, q_len, suffix, group_sizes, prefix, hq, hkv, d, page, seed=0, spread=1.0, spare=2, pad=0):
        import tenant_composite_lora_gb300 as tcl
        self.tcl = tcl
        g, r = gen_of(seed), np.random.RandomState(seed)
        self.q_len, self.suffix, self.prefix = list(q_len), list(suffix), list(prefix)
        self.go = np.concatenate([[0], np.cumsum(group_sizes)]).astype(int)
        self.hq, self.hkv, self.d, self.page = hq, hkv, d, page
        B, NG, self.TQ = len(q_len), len(group_sizes), int(sum(q_len))
        self.q_off = np.concatenate([[0], np.cumsum(q_len)]).astype(int)
        need = lambda n: -(-n // page)
        sp, pp = [need(n) for n in suffix], [need(n) for n in prefix]
        total = sum(sp) + sum(pp)
        self.pages = total + spare
        order = r.permutation(self.pages)
        self.s_tab = np.full((B, max(sp + [1])), self.pages + 9)  # unused entries name no page
        self.p_tab = np.full((max(NG, 1), max(pp + [1])), -5)
        at = 0
        for tab, counts in ((self.p_tab, pp), (self.s_tab, sp)):
            for i, n in enumerate(counts):
                tab[i, :n] = order[at:at + n]
                at += n
        nan = lambda: torch.full((self.pages, hkv, page, d), math.nan, dtype=torch.bfloat16, device="cuda")
        self.k, self.v = nan(), nan()
        self.ks, self.vs = {}, {}
        for kind, lens, tab in (("p", prefix, self.p_tab), ("s", suffix, self.s_tab)):
            for i, n in enumerate(lens):
                if n == 0:
                    continue
                kk, vv = (spread * rand(g, n, hkv, d).float()).to(torch.bfloat16), rand(g, n, hkv, d)
                self.ks[kind, i], self.vs[kind, i] = kk, vv
                j = torch.arange(n, device="cuda")
                pg = dev(tab[i], torch.int64)[j // page]
                self.k[pg, :, j % page] = kk
                self.v[pg, :, j % page] = vv
        row = hq * d
        self.q = rand(g, max(self.TQ, 1), row + pad)[:self.TQ, :row].view(self.TQ, hq, d)
        self.scale = d ** -0.5

    def run(self, stream=None, lse=True):
        tcl = self.tcl
        B, NG = len(self.q_len), len(self.go) - 1
        cache = tcl.LoraKvCache(self.pages, self.page, self.hkv, self.d, k=self.k, v=self.v)
        plan = tcl.LoraAttnPlan(max(B, 1), NG, max(self.TQ, 1), self.p_tab.shape[1], self.s_tab.shape[1], self.hq,
                                self.hkv, self.d, self.page)
        plan.build(dev(self.q_off), dev(self.suffix), dev(self.s_tab), self.TQ, self.pages,
                   dev(self.go) if NG else None, dev(self.prefix) if NG else None, dev(self.p_tab) if NG else None,
                   stream=stream)
        out = torch.full((self.TQ, self.hq, self.d), 3.0, dtype=torch.bfloat16, device="cuda")
        l = torch.full((self.TQ, self.hq), 3.0, device="cuda") if lse else None
        tcl.prefix_attention(self.q, cache, plan, self.scale, out=out, lse=l, stream=stream)
        self.status = plan.status(stream)
        return out, l

    def reference(self, hide=lambda kind, i, n: None):
        """(out, lse, sum p |v|, score error) in 64 bits."""
        G = self.hq // self.hkv
        shape = (self.TQ, self.hq)
        out = torch.zeros(*shape, self.d, dtype=torch.float64, device="cuda")
        mag, lse = torch.zeros_like(out), torch.full(shape, -math.inf, dtype=torch.float64, device="cuda")
        err = torch.zeros(shape, dtype=torch.float64, device="cuda")
        for b, n in enumerate(self.q_len):
            grp = int(np.searchsorted(self.go[1:], b, side="right")) if len(self.go) > 1 else -1
            for i in range(n):
                t, parts = self.q_off[b] + i, []
                if grp >= 0 and self.prefix[grp]:
                    parts.append(("p", grp, self.prefix[grp]))
                own = max(0, self.suffix[b] - n + i + 1)
                if own and self.suffix[b]:
                    parts.append(("s", b, own))
                if not parts:
                    continue
                k = torch.cat([self.ks[x, y][:m] for x, y, m in parts]).double()
                v = torch.cat([self.vs[x, y][:m] for x, y, m in parts]).double()
                seen = torch.cat([torch.ones(m, dtype=torch.bool, device="cuda") if hide(x, y, m) is None
                                  else hide(x, y, m) for x, y, m in parts])
                k, v = k[seen].repeat_interleave(G, 1), v[seen].repeat_interleave(G, 1)
                q = self.q[t].double()
                if not k.shape[0]:
                    continue
                s = torch.einsum("hd,khd->hk", q, k) * self.scale
                p = torch.softmax(s, -1)
                out[t] = torch.einsum("hk,khd->hd", p, v)
                mag[t] = torch.einsum("hk,khd->hd", p, v.abs())
                lse[t] = torch.logsumexp(s, -1)
                err[t] = (torch.einsum("hd,khd->hk", q.abs(), k.abs()) * abs(self.scale)).amax(-1) * 2.0 ** -17
        return out, lse, mag, err

    def check(self, out, lse, ref):
        r_out, r_lse, mag, err = ref
        tol = U * r_out.abs() + (U + 2 * err[..., None] + 2.0 ** -14) * mag
        off = (out.double() - r_out).abs()
        assert bool((off <= tol).all()), float((off - tol).max())
        if lse is not None:
            empty = r_lse == -math.inf
            assert bool((lse[empty] == -math.inf).all())
            d = (lse.double() - r_lse).abs()[~empty]
            assert bool((d <= (err + 2.0 ** -20 * (1 + r_lse.abs()))[~empty]).all()), float(d.max())


SHAPES = [(8, 2, 128, 16), (4, 4, 64, 32), (6, 2, 128, 64), (16, 1, 64, 16), (8, 8, 128, 128), (40, 1, 128, 32)]


@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
@pytest.mark.parametrize("prefix", [0, 1, 16, 127, 128, 129, 700])
def test_decode_matches_the_formula(hq, hkv, d, page, prefix):
    """Single tokens behind one prefix; own parts of one token to several tiles."""
    suffix = [1, 2, 15, 16, 17, 63, 64, 65, 130, 300]
    b = Batch([1] * len(suffix), suffix, [len(suffix)], [prefix], hq, hkv, d, page, seed=prefix + page)
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
def test_no_prefix_matches_the_formula(hq, hkv, d, page):
    b = Batch([1, 1, 1], [1, 200, 33], [], [], hq, hkv, d, page, seed=page)
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
def test_ragged_groups_and_empty_rows(hq, hkv, d, page):
    """Groups of 1 to many requests and one without any, prefixes of none to
    many tokens, requests without query tokens, rows that see no key."""
    q_len = [1, 0, 3, 1, 2, 1, 5, 1, 1, 4]
    suffix = [5, 9, 3, 0, 2, 40, 1, 150, 0, 30]  # requests 3 and 8 own nothing; 6 has fewer keys than queries
    b = Batch(q_len, suffix, [3, 1, 0, 4, 2], [300, 0, 77, 19, 0], hq, hkv, d, page, seed=1)
    out, lse = b.run()
    assert b.status == 0
    ref = b.reference()
    assert bool((ref[1] == -math.inf).any())
    b.check(out, lse, ref)


@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
@pytest.mark.parametrize("n", [2, 17, 130, 300])
def test_several_queries_are_causal(hq, hkv, d, page, n):
    """Verification of drafted tokens and prefill chunks: query i sees itself
    and what precedes it."""
    b = Batch([n, 1, n // 2], [n, 40, n // 2 + 170], [2, 1], [50, 260], hq, hkv, d, page, seed=n, pad=8)
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 128, 16), (4, 4, 64, 64)])
@pytest.mark.parametrize("groups", [1, 3])
def test_many_requests_behind_long_prefixes(hq, hkv, d, page, groups):
    """Row counts of several tiles, key axes that are split over the SMs."""
    B = 200
    r = np.random.RandomState(groups)
    sizes = [B] if groups == 1 else [150, 1, 49]
    b = Batch([1] * B, r.randint(0, 90, B), sizes, [3001] if groups == 1 else [2500, 4000, 129], hq, hkv, d, page)
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("d", [64, 128])
def test_one_request_with_a_long_context(d):
    b = Batch([1], [70001], [1], [30011], 8, 1, d, 32, seed=9)
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("spread", [8.0, 40.0])
def test_scores_that_grow_along_the_keys(spread):
    """Large scores of both signs, the largest late: the running maximum moves."""
    b = Batch([1] * 40 + [200], [20] * 40 + [200], [41], [900], 8, 2, 128, 16, seed=5, spread=spread)
    for kind, i, n in [("p", 0, 900)] + [("s", j, 20) for j in range(40)] + [("s", 40, 200)]:
        ramp = torch.linspace(0.05, 1.0, n, device="cuda")[:, None, None]
        b.ks[kind, i] = (b.ks[kind, i].float() * ramp).to(torch.bfloat16)
        tab = b.p_tab if kind == "p" else b.s_tab
        j = torch.arange(n, device="cuda")
        b.k[dev(tab[i], torch.int64)[j // 16], :, j % 16] = b.ks[kind, i]
    out, lse = b.run()
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("hq,hkv,d,page", SHAPES)
@pytest.mark.parametrize("scale", [-0.2, 0.0])
def test_scales_that_are_not_positive(hq, hkv, d, page, scale):
    b = Batch([1] * 20 + [70], [3] * 10 + [50] * 10 + [90], [21], [400], hq, hkv, d, page, seed=6)
    b.scale = scale
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("hq,hkv,d,page", [(8, 2, 128, 16), (4, 4, 64, 64)])
@pytest.mark.parametrize("q_len,suffix,sizes,prefix", [
    ([1] * 90, [400] * 90, [60, 30], [1, 0]),             # one short wide segment a head beside a cache full of narrow ones
    ([300, 260, 1], [2100, 2600, 1], [3], [40]),          # one narrow segment of a key
    ([1] * 70 + [200], [0] * 70 + [200], [71], [2000]),   # wide ones alone
    ([1] * 12, [900] * 12, [1] * 12, [700] * 12),         # narrow ones alone
])
def test_mixtures_of_few_and_many_rows(hq, hkv, d, page, q_len, suffix, sizes, prefix):
    """The SMs are shared out between segments of few and of many rows, down to one SM for either."""
    b = Batch(q_len, suffix, sizes, prefix, hq, hkv, d, page, seed=8)
    out, lse = b.run()
    assert b.status == 0
    b.check(out, lse, b.reference())


@pytest.mark.parametrize("n", [3, 40, 200])
def test_later_tokens_do_not_reach_earlier_queries(n):
    """A later token's key and value of inf or NaN leave the queries before it unchanged."""
    b = Batch([n], [n + 21], [1], [33], 8, 2, 128, 16, seed=n)
    clean, clean_lse = b.run()
    at = n + 21 - n + n // 2  # seen by queries n // 2 and later
    j = torch.arange(at, n + 21, device="cuda")
    pg = dev(b.s_tab[0], torch.int64)[j // 16]
    bad = torch.tensor([math.inf, -math.inf, math.nan], dtype=torch.bfloat16, device="cuda")
    b.v[pg, :, j % 16] = bad[torch.randint(0, 3, (j.numel(), 2, 128), device="cuda")]
    out, lse = b.run()
    torch.cuda.synchronize()
    assert torch.equal(out[:n // 2], clean[:n // 2]) and torch.equal(lse, clean_lse)
    assert not bool(torch.isfinite(out[n // 2:]).any())
    b.k[pg, :, j % 16] = math.nan
    out, lse = b.run()
    assert torch.equal(out[:n // 2], clean[:n // 2]) and torch.equal(lse[:n // 2], clean_lse[:n // 2])
    assert bool(torch.isnan(out[n // 2:]).all())


def test_strided_tokens_another_stream_and_no_lse():
    """q a slice of a wider buffer, out of one too, on a stream of the user's."""
    b = Batch([1, 4, 1], [90, 30, 7], [2, 1], [200, 10], 8, 2, 128, 16, seed=2, pad=264)
    assert b.q.stride(0) == 8 * 128 + 264
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out, lse = b.run(stream=st)
    st.synchronize()
    b.check(out, lse, b.reference())
    only, none = b.run(lse=False)
    assert none is None and torch.equal(only, out)


def test_runs_are_alike_bit_for_bit_and_inside_a_graph():
    import tenant_composite_lora_gb300 as tcl
    b = Batch([1] * 30 + [40], [33] * 30 + [60], [31], [1500], 8, 2, 128, 16, seed=8)
    first = b.run()
    again = b.run()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # the build and the attention as a captured graph, replayed on other lengths
    cache = tcl.LoraKvCache(b.pages, 16, 2, 128, k=b.k, v=b.v)
    plan = tcl.LoraAttnPlan(31, 1, b.TQ, b.p_tab.shape[1], b.s_tab.shape[1], 8, 2, 128, 16)
    t = [dev(x) for x in (b.q_off, b.suffix, b.s_tab, b.go, b.prefix, b.p_tab)]
    out, lse = torch.zeros_like(first[0]), torch.zeros_like(first[1])

    def step():
        plan.build(t[0], t[1], t[2], b.TQ, b.pages, t[3], t[4], t[5])
        tcl.prefix_attention(b.q, cache, plan, b.scale, out=out, lse=lse)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    b.suffix = [7] * 30 + [41]
    b.prefix = [777]
    t[1].copy_(dev(b.suffix))
    t[4].copy_(dev(b.prefix))
    b.ks = {key: x[:777 if key[0] == "p" else b.suffix[key[1]]] for key, x in b.ks.items()}
    b.vs = {key: x[:777 if key[0] == "p" else b.suffix[key[1]]] for key, x in b.vs.items()}
    graph.replay()
    torch.cuda.synchronize()
    b.check(out, lse, b.reference())


def test_cache_beyond_32_bit_offsets():
    """Keys and values beyond 2^32 elements (8 GB) from the cache's start."""
    import tenant_composite_lora_gb300 as tcl
    page, hkv, d, hq = 128, 8, 128, 8
    pages = (1 << 32) // (page * hkv * d) + 40
    k = torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    small = Batch([1, 1], [300, 20], [2], [500], hq, hkv, d, page, seed=3)
    n = small.pages
    k[pages - n:], v[pages - n:] = small.k, small.v
    small.k, small.v, small.pages = k, v, pages
    small.s_tab, small.p_tab = small.s_tab + pages - n, small.p_tab + pages - n
    out, lse = small.run()
    small.check(out, lse, small.reference())
    # and an append there
    cache = tcl.LoraKvCache(pages, page, hkv, d, k=k, v=v)
    new = rand(gen_of(1), 1, hkv, d)
    tcl.kv_append(cache, new, new, dev([pages * page - 1]))
    torch.cuda.synchronize()
    assert torch.equal(k[pages - 1, :, page - 1], new[0]) and torch.equal(v[pages - 1, :, page - 1], new[0])


def test_malformed_batches_set_status_bits():
    import tenant_composite_lora_gb300 as tcl
    n = tcl.native

    def fresh():
        return Batch([1, 1, 2], [20, 33, 40], [2, 1], [50, 18], 4, 2, 64, 16, seed=6)

    b = fresh()  # a page id outside the cache hides that page's keys
    b.s_tab[1, 1], b.p_tab[0, 0] = b.pages, -1
    out, lse = b.run()
    assert b.status == n.LORA_DEV_BAD_PAGE

    def hide(kind, i, m):
        seen = torch.ones(m, dtype=torch.bool, device="cuda")
        if (kind, i) == ("s", 1):
            seen[16:32] = False
        if (kind, i) == ("p", 0):
            seen[:16] = False
        return seen

    b.check(out, lse, b.reference(hide))
    for field, at, value in (("suffix", 1, -3), ("suffix", 1, 10 ** 6), ("prefix", 0, -1), ("prefix", 0, 10 ** 6)):
        b = fresh()
        getattr(b, field)[at] = value
        out, lse = b.run()
        assert b.status == n.LORA_DEV_BAD_LENGTH
        getattr(b, field)[at] = 0  # counts as 0
        b.check(out, lse, b.reference())
    b = fresh()  # malformed row pointers: no batch; no prefixes
    b.q_off[1] = 3
    out, lse = b.run()
    assert b.status == n.LORA_DEV_BAD_LENGTH
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    b = fresh()
    b.go[1] = 4
    out, lse = b.run()
    assert b.status == n.LORA_DEV_BAD_LENGTH
    b.go = np.array([0])
    b.check(out, lse, b.reference())


def test_attention_refuses_what_it_cannot_take():
    import tenant_composite_lora_gb300 as tcl
    b = Batch([1, 1], [20, 33], [2], [50], 4, 2, 64, 16, seed=6)
    cache = tcl.LoraKvCache(b.pages, 16, 2, 64, k=b.k, v=b.v)
    plan = tcl.LoraAttnPlan(2, 1, 2, 4, 3, 4, 2, 64, 16)
    with pytest.raises(tcl.LoraError):  # not built
        tcl.lora_prefix_attention(b.q.data_ptr(), 256, b.q.data_ptr() + 4096, 256, None, cache.handle, plan.handle, 1.0)
    args = (dev(b.q_off), dev(b.suffix), dev(b.s_tab), 2, b.pages, dev(b.go), dev(b.prefix), dev(b.p_tab))
    with pytest.raises(tcl.LoraError):  # more requests than the plan takes
        plan.build(dev([0, 1, 2, 2]), dev([1, 1, 1]), dev(np.zeros((3, 1))), 2, b.pages)
    with pytest.raises(tcl.LoraError):  # more query tokens
        plan.build(args[0], args[1], args[2], 3, b.pages)
    with pytest.raises(ValueError, match="2 requests"):
        plan.build(args[0], args[1][:1], args[2], 2, b.pages)
    plan.build(*args)
    out = torch.empty_like(b.q)
    with pytest.raises(ValueError, match="q: shape"):
        tcl.prefix_attention(b.q[:1], cache, plan, out=out)
    with pytest.raises(ValueError, match="lse must hold"):
        tcl.prefix_attention(b.q, cache, plan, out=out, lse=torch.zeros(3, device="cuda"))
    with pytest.raises(tcl.LoraError):  # out is q
        tcl.prefix_attention(b.q, cache, plan, out=b.q)
    with pytest.raises(tcl.LoraError):  # a cache with fewer pages than the build was checked against
        tcl.prefix_attention(b.q, tcl.LoraKvCache(b.pages - 1, 16, 2, 64), plan, out=out)
    with pytest.raises(tcl.LoraError):  # another layout
        tcl.prefix_attention(b.q, tcl.LoraKvCache(b.pages, 32, 2, 64), plan, out=out)
    tcl.prefix_attention(b.q, cache, plan, out=out)
    for bad in ((0, 1, 1, 1, 1, 4, 2, 64, 16), (1, 1, 1, 1, 1, 5, 2, 64, 16), (1, 1, 1, 1, 1, 4, 2, 80, 16),
                (1, 1, 1, 1, 1, 4, 2, 64, 48), (1, -1, 1, 1, 1, 4, 2, 64, 16)):
        with pytest.raises(tcl.LoraError):
            tcl.LoraAttnPlan(*bad)
