"""Token sampling against its definition in 64 bits.

The expected token does not hinge on rounding: each u lies in the middle of a
token's interval of the kept mass, top_p in the middle between two cumulated
masses, and the intervals are far wider (1e-4 and up) than the error of a
32-bit exp (about 1e-6); min_p is as far from the weights.  A probability is
a 32-bit exp over a sum: 4e-6 relative (its argument, at most 30, rounded to
2^-24 of it, and the last bits).
"""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    from tenant_composite_lora_gb300 import build
    build.build()


def ordered(l):
    """Indices by (logit descending, index ascending), without those of no weight."""
    l = np.where(np.isnan(l), -np.inf, l)
    order = np.argsort(-l, kind="stable")
    return order[l[order] > -np.inf]


def kept(l, tau=1.0, k=0, p=1.0, mp=0.0):
    """(indices of the kept tokens ascending, their weights)."""
    order = ordered(l)
    if tau <= 0:
        order, tau = order[:1], 1.0
    if 0 < k:
        order = order[:k]
    top = l[order[0]]
    with np.errstate(invalid="ignore"):
        e = np.where(l[order] == top, 1.0, np.exp((l[order] - top) / tau))
    before = np.concatenate([[0.0], np.cumsum(e)[:-1]])
    keep = (np.arange(e.size) == 0) | (((before < p * e.sum()) | (p >= 1)) & (e >= min(mp, 1.0)))
    order, e = order[keep], e[keep]
    by = np.argsort(order)
    return order[by], e[by]


def middle_p(l, tau, k, frac):
    """A top_p in the middle of the interval that ends the prefix of about `frac` of the mass."""
    order = ordered(l)
    order = order[:k] if k > 0 else order
    e = np.exp((l[order] - l[order[0]]) / tau)
    c = np.cumsum(e) / e.sum()
    width = np.diff(np.concatenate([[0.0], c]))
    wide = np.flatnonzero(width > 2e-4)
    at = wide[np.argmin(np.abs(c[wide] - frac))]
    return float(c[at] - width[at] / 2)


def middle_min_p(l, tau, near=0.0437):
    """A min_p between two weights that are far apart (2e-5), about `near`."""
    e = np.unique(np.exp((l[ordered(l)] - l[ordered(l)[0]]) / tau))
    gaps = np.flatnonzero(np.diff(e) > 2e-5)
    if not gaps.size:
        return near
    at = gaps[np.argmin(np.abs(e[gaps] - near))]
    return float(e[at] + e[at + 1]) / 2


def middle_u(e, r):
    """u in the middle of the interval of a token that is wide enough."""
    share = e / e.sum()
    at = r.choice(np.flatnonzero(share > min(1e-4, share.max() * 0.99)))
    return float(np.cumsum(share)[at] - share[at] / 2), at


def run(logits, u, tau=None, k=None, p=None, mp=None):
    import tenant_composite_lora_gb300 as tcl
    T = logits.shape[0]
    f = lambda x: None if x is None else torch.as_tensor(np.asarray(x, np.float32)).cuda()
    probs = torch.full((T,), -1.0, device="cuda")
    tok = tcl.sample(logits, f(u), f(tau), None if k is None else torch.as_tensor(np.asarray(k, np.int32)).cuda(),
                     f(p), f(mp), probs=probs)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), probs.cpu().numpy().astype(np.float64)


def as_seen(l, dtype):
    t = torch.as_tensor(l.astype(np.float32)).to(dtype)
    return t.cuda(), t.double().numpy()


def expect(logits, seen, rows):
    """rows: (tau, k, p, mp) per row; draws u, runs, compares tokens and shares."""
    r = np.random.RandomState(7)
    us, toks, shares = [], [], []
    for l, (tau, k, p, mp) in zip(seen, rows):
        idx, e = kept(l, tau, k, p, mp)
        u, at = middle_u(e, r)
        us.append(u)
        toks.append(idx[at])
        shares.append(e[at] / e.sum())
    got, prob = run(logits, us, *map(list, zip(*rows)))
    np.testing.assert_array_equal(got, toks)
    np.testing.assert_allclose(prob, shares, rtol=4e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 31, 1000, 4097, 32768, 131001])
def test_settings_match_the_definition(V, dtype):
    r = np.random.RandomState(V)
    rows, ls = [], []
    for frac in (None, 0.3, 0.9, 0.99):
        for k in (0, 1, 7, 50, 1000, V):
            for tau in (0.6, 1.0, 1.7):
                ls.append(r.randn(V) * 2.5)
                ls[-1][r.randint(0, V, 20)] += r.uniform(2, 9, 20)
                rows.append([tau, k, frac])
    logits, seen = as_seen(np.stack(ls), dtype)
    rows = [(np.float32(tau), k, 1.0 if frac is None else np.float32(middle_p(l, np.float32(tau), k, frac)),
             0.0 if i % 3 else np.float32(middle_min_p(l, np.float32(tau)))) for i, ((tau, k, frac), l) in enumerate(zip(rows, seen))]
    expect(logits, seen, [tuple(float(x) if j != 1 else x for j, x in enumerate(row)) for row in rows])


@pytest.mark.parametrize("V", [300, 5000, 70000])
def test_ties_go_by_index(V):
    """Logits of a few levels: top_k and top_p cut through equal logits."""
    r = np.random.RandomState(V)
    base = np.log(np.array([1.0, 1.0, 0.5, 0.25, 0.125]))
    ls = base[r.randint(0, 5, (24, V))].astype(np.float32)
    rows = []
    for i in range(24):
        k = [0, 1, 5, V // 7, V // 2, V - 3][i % 6]
        e = np.exp(ls[i].astype(np.float64))[ordered(ls[i].astype(np.float64))]
        e = e[:k] if k else e
        # a top_p in the middle of a tie's interval (at least 1 / (8 V) wide, so exact sums are needed)
        c = np.cumsum(e)
        at = r.randint(e.size)
        p = 1.0 if i % 4 == 0 else float(np.float32((c[at] - e[at] / 2) / c[-1]))
        if p < 1.0 and abs(p * c[-1] - (c[at] - e[at] / 2)) > e[at] / 4:  # the float32 is too coarse for it
            p = 1.0
        rows.append((1.0, k, p, 0.0))
    us, toks = [], []
    for l, (tau, k, p, mp) in zip(ls.astype(np.float64), rows):
        idx, e = kept(l, tau, k, p, mp)
        share = e / e.sum()
        at = idx.size - 1 if p == 1.0 or k == 1 else r.randint(idx.size)  # the last kept token: the cut itself
        u = np.float32(np.cumsum(share)[at] - share[at] / 2)
        us.append(u)
        toks.append(idx[at])
    got, prob = run(torch.as_tensor(ls).cuda(), us, *map(list, zip(*rows)))
    np.testing.assert_array_equal(got, toks)


def test_greedy_takes_the_lowest_of_the_largest():
    l = np.full((4, 1000), -3.0)
    l[0, [700, 13, 950]] = 2.0
    l[1, 999] = 1.0
    l[2, 0] = 1.0
    l[3] = 0.0
    l[3, ::2] = -0.0  # equal to 0
    for dtype in (torch.float32, torch.bfloat16):
        logits, _ = as_seen(l, dtype)
        for tau in (0.0, -1.0, math.nan):
            got, prob = run(logits, [0.99] * 4, [tau] * 4, [0, 5, 0, 0], [0.5] * 4, [0.1] * 4)
            assert got.tolist() == [13, 999, 0, 0] and prob.tolist() == [1.0] * 4


def test_rows_with_masks_infinities_and_nan():
    V = 4000
    r = np.random.RandomState(1)
    l = r.randn(8, V).astype(np.float32)
    l[0] = -np.inf                                  # nothing to choose
    l[1] = np.nan
    l[2, :] = -np.inf
    l[2, 3210] = -50.0                              # one token left
    l[3, r.rand(V) < 0.95] = -np.inf                # a grammar's mask
    l[4] = np.where(r.rand(V) < 0.9, np.finfo(np.float32).min, l[4])  # a mask of the type's lowest value
    l[5] = np.finfo(np.float32).min                 # every token at the lowest value: all alike
    l[6, [17, 3001]] = np.inf                       # share the mass
    l[7, ::3] = np.nan                              # count as -inf
    rows = [(1.0, 0, 1.0, 0.0)] * 8
    us, toks = [0.5, 0.5], [-1, -1]
    for x in l[2:].astype(np.float64):
        idx, e = kept(x)
        u, at = middle_u(e, r)
        us.append(u)
        toks.append(idx[at])
    got, prob = run(torch.as_tensor(l).cuda(), us, *map(list, zip(*rows)))
    np.testing.assert_array_equal(got, toks)
    assert prob[0] == prob[1] == 0.0 and prob[2] == 1.0 and prob[6] == 0.5
    got, _ = run(torch.as_tensor(l).cuda(), us, [1.0] * 8, [40] * 8, [0.9] * 8, [0.05] * 8)
    assert got[:2].tolist() == [-1, -1] and got[2] == 3210
    assert all(np.isfinite(l[i, got[i]]) for i in (3, 7)) and got[6] in (17, 3001)


def test_edges_of_u_and_of_the_settings():
    l = np.log(np.array([[0.2, 0.0, 0.3, 0.5, 0.0]] * 6, dtype=np.float32) + 1e-30).astype(np.float32)
    l[:, 1] = -np.inf
    l[:, 4] = -np.inf
    logits = torch.as_tensor(l).cuda()
    got, _ = run(logits, [0.0, np.nextafter(np.float32(1), np.float32(0)), 1.0, 2.0, -1.0, math.nan])
    assert got.tolist() == [0, 3, 3, 3, 0, 0]  # outside [0, 1): the nearest kept token
    # top_p <= 0 and min_p >= 1 leave the largest; NaN settings and a negative k are off; k above V is off
    u = [0.1] * 6
    assert run(logits, u, p=[0.0, -1.0] * 3)[0].tolist() == [3] * 6
    assert run(logits, u, mp=[1.0, 5.0] * 3)[0].tolist() == [3] * 6
    assert run(logits, u, p=[math.nan] * 6, mp=[math.nan] * 6, k=[-4, 9] * 3)[0].tolist() == [0] * 6
    assert run(logits, u)[0].tolist() == [0] * 6
    # tiny and huge temperatures
    assert run(logits, u, tau=[1e-42, 1e-30, 1e-3] * 2)[0].tolist() == [3] * 6
    assert run(logits, [0.1, 0.4, 0.9] * 2, tau=[math.inf] * 6)[0].tolist() == [0, 2, 3] * 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_strided_unaligned_rows_and_another_stream(dtype):
    import tenant_composite_lora_gb300 as tcl
    r = np.random.RandomState(3)
    big, seen = as_seen(r.randn(9, 5001) * 3, dtype)
    for c0 in (0, 1, 3):
        rows = [(1.0, 30, 1.0, 0.0)] * 9
        expect(big[:, c0:c0 + 4093], seen[:, c0:c0 + 4093], rows)
    u = torch.rand(9, device="cuda")
    here = tcl.sample(big, u)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    there = tcl.sample(big, u, stream=st)
    st.synchronize()
    assert torch.equal(here, there)
    assert tcl.sample(big[:0], u).numel() == 0


@pytest.mark.parametrize("T,V", [(1, 131072), (3, 1 << 20), (700, 257), (150, 50001)])
def test_batches_of_few_and_many_rows(T, V):
    r = np.random.RandomState(T)
    logits, seen = as_seen(r.randn(T, V) * (1.0 if V < 1000 else 4.0), torch.float32)
    expect(logits, seen, [(0.8, 0 if t % 2 else 64, 1.0, 0.0) for t in range(T)])


def test_nearly_flat_rows_keep_most_of_the_vocabulary():
    """Cuts that keep tens of thousands of nearly equal tokens: the kept set itself, seen through u at its ends."""
    V = 60000
    r = np.random.RandomState(11)
    l = (r.randn(6, V) * 1e-3).astype(np.float32)
    for k, cut in ((30000, 30000), (0, 42000), (45000, 22500)):
        us, toks, ps = [], [], []
        for row, last in zip(l.astype(np.float64), [True, False] * 3):
            e = np.exp(row[ordered(row)] - row.max())[:k or V]
            # top_p in the middle of token cut - 1: half a token's mass is 1e-5, the sums are good to 1e-7
            p = 1.0 if cut == k else float(np.float32((e[:cut - 1].sum() + e[cut - 1] / 2) / e.sum()))
            idx, _ = kept(row, 1.0, k, p)
            assert idx.size == cut
            us.append(1.0 if last else 0.0)
            toks.append(idx[-1] if last else idx[0])
            ps.append(p)
        got, prob = run(torch.as_tensor(l).cuda(), us, None, [k] * 6, ps)
        np.testing.assert_array_equal(got, toks)
        np.testing.assert_allclose(prob, [1.0 / cut] * 6, rtol=1e-2)  # (one token more or fewer shows above)


def wide_enough(share):
    """For long rows: tokens of 4e-6 of the mass and up, or 0.99 of the largest (at least 1.8e-6 here).  Half of that
    is above 9e-7; the sums' error is below 5e-7 of the mass (a weight's 2^-22, sums of at most 32 in 32 bits)."""
    return np.flatnonzero(share > min(4e-6, share.max() * 0.99))


def middle_of_wide(l, tau, k, frac):
    order = ordered(l)
    order = order[:k] if k > 0 else order
    e = np.exp((l[order] - l[order[0]]) / tau)
    c = np.cumsum(e) / e.sum()
    width = np.diff(np.concatenate([[0.0], c]))
    wide = wide_enough(width)
    at = wide[np.argmin(np.abs(c[wide] - frac))]
    return float(c[at] - width[at] / 2)


@pytest.mark.parametrize("T,V,dtype", [(256, 131001, torch.bfloat16), (240, 40000, torch.float32),
                                       (3, 600001, torch.bfloat16), (5, (1 << 19) + 5, torch.float32)])
def test_many_or_very_long_rows_end_at_the_cut(T, V, dtype):
    """Rows in descending order, so that a u near 1 gives the cut itself."""
    r = np.random.RandomState(T)
    ls, rows = [], []
    for t in range(T):
        kind = t % 10
        l = r.randn(V) * (2.5 if kind in (0, 1, 6) else 0.4)
        if kind == 3:
            l[:] = 1.25  # all alike
        elif kind == 4:
            l = np.where(r.rand(V) < 0.5, 0.0, -1.0)  # two values
        elif kind == 5:
            l[r.rand(V) < 0.9] = -np.inf
        elif kind == 6:
            l[:30] += 9
        elif kind == 9:
            l = r.randn(V) * 0.02
        ls.append(-np.sort(-np.round(l * 256) / 256))
        k = {7: 3000, 8: V // 2}.get(kind, 0)
        rows.append((float(np.float32(r.uniform(0.5, 1.3))), k, [0.95, 0.8, 0.5, 0.999, 1.0][r.randint(5)],
                     kind in (2, 6)))
    logits, seen = as_seen(np.stack(ls), dtype)
    settings, us, toks, shares = [], [], [], []
    for l, (tau, k, frac, with_mp) in zip(seen, rows):
        p = 1.0 if frac == 1.0 else float(np.float32(middle_of_wide(l, tau, k, frac)))
        mp = float(np.float32(middle_min_p(l, tau, near=0.3))) if with_mp else 0.0
        idx, e = kept(l, tau, k, p, mp)
        share = e / e.sum()
        at = wide_enough(share)[-1]
        settings.append((tau, k, p, mp))
        us.append(float(np.cumsum(share)[at] - share[at] / 2))
        toks.append(idx[at])
        shares.append(share[at])
    got, prob = run(logits, us, *map(list, zip(*settings)))
    np.testing.assert_array_equal(got, toks)
    np.testing.assert_allclose(prob, shares, rtol=4e-6)


def test_sample_refuses_what_it_cannot_take():
    import tenant_composite_lora_gb300 as tcl
    l, u = torch.zeros(4, 32, device="cuda"), torch.zeros(4, device="cuda")
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        tcl.sample(l.half(), u)
    with pytest.raises(ValueError, match="must be contiguous"):
        tcl.sample(torch.zeros(32, 4, device="cuda").t(), u)
    with pytest.raises(ValueError, match="u holds 3"):
        tcl.sample(l, u[:3])
    with pytest.raises(ValueError, match="top_k: int32"):
        tcl.sample(l, u, top_k=u)
    with pytest.raises(ValueError, match="a CUDA tensor"):
        tcl.sample(l.cpu(), u)
    tok = torch.zeros(4, dtype=torch.int32, device="cuda")
    for kind, stride, V in ((2, 32, 32), (0, 31, 32), (0, 32, 0)):
        with pytest.raises(tcl.LoraError) as e:
            tcl.lora_sample(l.data_ptr(), kind, stride, 4, V, u, None, None, None, None, tok)
        assert e.value.status == tcl.native.LORA_ERR_INVALID_ARG
    with pytest.raises(tcl.LoraError) as e:
        tcl.lora_sample(l.data_ptr(), 0, (1 << 20) + 1, 4, (1 << 20) + 1, u, None, None, None, None, tok)
    assert e.value.status == tcl.native.LORA_ERR_NOT_SUPPORTED
