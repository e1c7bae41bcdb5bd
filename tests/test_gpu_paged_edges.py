"""The paged cache's calls at their edges: rows that nothing writes, infinities and NaN, scales at the
ends of their range.  References and tolerances are those of test_gpu_paged.py."""
import numpy as np
import pytest
import torch

import paged_plain as plain
from test_gpu_paged import FP8, _cache, _check_attn, _freq, _new, _rows, _state, lsa

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("B,Nq,Hq", [(3, 1, 8), (4, 40, 24), (500, 17, 4)])
def test_append_leaves_no_row_of_a_new_tensor_unwritten(compiled, B, Nq, Hq, monkeypatch):
    # rows of padding and of a sequence with a negative start are zeros in a new tensor, whose
    # memory held NaN; in a given one padding stays and the left-out sequence becomes zeros; in
    # place both stay.  One, several and no CTAs of the queries' own.
    if not compiled:
        monkeypatch.setattr(lsa, "_binding", None)
    rng = np.random.default_rng(7)
    Hkv, d, page = 2, 64, 16
    c = lsa.LsaPagedKV.empty(B, B * 4 + 1, page, 4, Hkv, d, FP8)
    c.page_table.copy_(torch.arange(B * 4, dtype=torch.int32).view(B, 4))
    k, q = _new(rng, B, Nq, Hkv, d).cuda(), _new(rng, B, Nq, Hq, d).cuda()
    start = torch.full((B,), 5, dtype=torch.int32, device="cuda")
    start[1] = -1
    n_new = torch.full((B,), Nq, dtype=torch.int32, device="cuda")
    n_new[0], n_new[2] = Nq // 2, 0
    inv = torch.from_numpy(_freq(64)).cuda()

    def call(**kw):
        return lsa.lsa_paged_append(c, k, k, start, inv_freq=inv, **kw)

    want = call(n_new=n_new, q=q.clone(), q_out=torch.zeros_like(q))     # rotated; zeros elsewhere
    assert (want[3:].float().abs().amax((1, 2, 3)) > 0).all()
    for with_n in (True, False):
        nan = [torch.full_like(q, float("nan")) for _ in range(8)]       # (memory to be given again)
        del nan
        got = call(n_new=n_new if with_n else None, q=q)
        assert torch.isfinite(got).all()
        assert (got[1] == 0).all()
        if with_n:
            assert torch.equal(got, want)
        del got
    sevens = torch.full_like(q, 7.0)
    call(n_new=n_new, q=q, q_out=sevens)
    assert (sevens[1] == 0).all() and (sevens[0, Nq // 2:] == 7).all() and (sevens[2] == 7).all()
    assert torch.equal(sevens[3:], want[3:])
    mine = q.clone()
    call(n_new=n_new, q=mine, q_out=mine)
    assert torch.equal(mine[1], q[1]) and torch.equal(mine[2], q[2])
    assert torch.equal(mine[3:], want[3:])
    with pytest.raises(lsa.LsaError):
        c.check()                                        # the negative start


# few units (clusters of several CTAs), many (a CTA each), more than one launch
SPLITS = [(1, 3, 700), (1, 420, 60), (1, 300, 1100)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("B,Nq,s", SPLITS)
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_attention_with_a_query_that_is_not_finite(dtype, B, Nq, s, bad):
    # every logit of that head is an infinity or NaN, all of them -inf for some: its results are
    # NaN, never those of an empty row; other heads and rows do not notice, and a row without a
    # key stays empty
    rng = np.random.default_rng(101)
    Hq, Hkv, d, page, mp = 8, 2, 64, 16, 30
    c = _cache(rng, B, Hkv, d, page, mp, dtype)
    if dtype == FP8:
        c.k_pages.view(torch.uint8).bitwise_and_(0x7F)  # (no key's sign differs)
    else:
        c.k_pages.abs_()
    idx, cnt = _rows(rng, B, Nq, mp * page, s, [s, 1, s, 0, 17])
    cnt[0, 2] = 5
    idx[0, 2, :5] = -1                                  # only positions that are skipped
    Q = _new(rng, B, Nq, Hq, d)
    Q[:, :, 3] = Q[:, :, 3].abs()                       # one head: all logits of one sign
    Q[:, :, 3, 7], Q[:, :, 6, 50] = bad, bad
    O, l = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                              return_lse=True)
    with pytest.raises(lsa.LsaError):
        c.check()                                       # the skipped positions
    full = torch.from_numpy(cnt > 0)
    full[0, 2] = False
    for h in (3, 6):
        assert torch.isnan(O[:, :, h].cpu()[full]).all() and torch.isnan(l[:, :, h].cpu()[full]).all()
    empty = ~full
    assert (O.cpu()[empty] == 0).all() and torch.isneginf(l.cpu()[empty]).all()
    fine = [0, 1, 2, 4, 5, 7]                           # (three of each KV head's four)
    some = np.arange(min(Nq, 12))
    _check_attn(c, Q[:, some][:, :, fine], idx[:, some], cnt[:, some], 1 / np.sqrt(d),
                O[:, some][:, :, fine], l[:, some][:, :, fine])


@pytest.mark.parametrize("dtype,bad", [(torch.bfloat16, float("inf")), (torch.bfloat16, float("-inf")),
                                       (torch.bfloat16, float("nan")), (FP8, float("nan"))])
@pytest.mark.parametrize("B,Nq,s", SPLITS)
@pytest.mark.parametrize("which", ["K", "V"])
def test_attention_over_a_listed_row_that_is_not_finite(dtype, bad, B, Nq, s, which):
    # a key's element: every head of its KV head is NaN in the rows that list it, whatever the
    # sign of the product; a value's element: that element is, and lse is not; rows that do not
    # list it, the other KV head and the other elements do not notice
    rng = np.random.default_rng(103)
    Hq, Hkv, d, page, mp = 8, 2, 128, 16, 30
    c = _cache(rng, B, Hkv, d, page, mp, dtype)
    clean = _state(c)
    idx, cnt = _rows(rng, B, Nq, mp * page - 1, s, [s, 1, s, 0, 17])    # (the last position in none)
    T = mp * page - 1
    hit = np.zeros((B, Nq), bool)
    for b in range(B):
        for i in range(0, Nq, 3):
            if cnt[b, i] > 0:
                idx[b, i, rng.integers(cnt[b, i])] = T
                hit[b, i] = True
    pages = c.k_pages if which == "K" else c.v_pages
    for b in range(B):
        pg = c.page_table[b, T // page]
        if dtype == FP8:
            pages.view(torch.uint8)[pg, T % page, 1, 9] = 0x7F
        else:
            pages[pg, T % page, 1, 9] = bad
    Q = _new(rng, B, Nq, Hq, d)
    O, l = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                              return_lse=True)
    c.check()
    O, l, hit = O.cpu(), l.cpu(), torch.from_numpy(hit)
    assert hit.any() and (~hit).any()
    if which == "K":
        assert torch.isnan(O[:, :, 4:][hit]).all() and torch.isnan(l[:, :, 4:][hit]).all()
    else:
        assert (~torch.isfinite(O[:, :, 4:, 9][hit])).all()
    # against the clean cache everywhere else
    st = dict(clean)
    Kv, Vv = st["K"], st["V"]
    sV = None
    if st["scales"] is not None:
        sc = np.repeat(st["scales"], plain.BLOCK, axis=1)
        Kv, Vv, sV = Kv * sc[:, :, 0, :, None], Vv * sc[:, :, 1, :, None], sc[:, :, 1]
    some = np.arange(min(Nq, 13))
    ro, ra, rz, rl = plain.attend(Kv, Vv, st["table"], Q[:, some].float().double().numpy(),
                                  idx[:, some], cnt[:, some], 1 / np.sqrt(d), sV)
    ra, floor = ra if sV is not None else (ra, 0.0)
    dz = 2.0 ** -18 * rz
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 4 * dz)[..., None] * ra + 2.0 ** -31 * floor + 1e-38
    skip = np.zeros(ro.shape, bool)
    rows = hit[:, some].numpy()
    if which == "K":
        skip[:, :, 4:] = rows[..., None, None]
    else:
        skip[:, :, 4:, 9] = rows[..., None]
    go = O[:, some].double().numpy()
    assert (np.abs(go - ro) <= tol)[~skip].all()
    gl = l[:, some].double().numpy()
    ok = ~np.isneginf(rl) & ~(skip.all(-1))
    assert (np.abs(gl[ok] - rl[ok]) <= (2 * dz + 2.0 ** -19 * (1 + np.abs(rl)))[ok]).all()
    assert np.array_equal(np.isneginf(gl), np.isneginf(rl))


@pytest.mark.parametrize("B,Nq,s", SPLITS)
def test_attention_logits_past_the_range_of_fp32(B, Nq, s):
    # logits that only the scale takes past the range: -inf beside others weighs nothing, and a row
    # of nothing else is no empty row
    rng = np.random.default_rng(107)
    Hq, Hkv, d, page, mp = 4, 1, 64, 16, 8
    c = _cache(rng, B, Hkv, d, page, mp, torch.bfloat16)
    c.k_pages.zero_()
    far = c.page_table[:, 0].long()
    c.k_pages[far] = 1e18                               # positions 0 .. 15: products of -6.4e36
    Q = torch.full((B, Nq, Hq, d), -1e17, dtype=torch.bfloat16)
    idx, cnt = _rows(rng, B, Nq, mp * page - page, s, [s, 1, s, 17])
    idx[idx >= 0] += page                               # of the other pages: logits of 0
    v = c.v_pages.float().cpu()
    idx[0, 0, 3], idx[0, 0, s - 1] = 4, 11              # two far ones in a full row
    idx[0, 1, 0] = 7                                    # a far one alone
    O, l = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                              scale=1e4, return_lse=True)
    c.check()
    assert torch.isnan(O[0, 1]).all() and torch.isneginf(l[0, 1]).all()
    table = c.page_table.cpu().numpy()
    t = np.delete(idx[0, 0, :s], [3, s - 1])
    want = v[table[0, t // page], t % page, 0].double().mean(0)
    size = v[table[0, t // page], t % page, 0].double().abs().mean(0)
    got = O[0, 0].cpu().double()
    assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -10 * size).all()
    assert ((l[0, 0].cpu().double() - np.log(len(t))).abs() <= 2.0 ** -19 * (1 + np.log(len(t)))).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("inter", [False, True])
def test_append_rotates_keys_and_queries_that_are_not_finite(dtype, inter):
    # an infinity's pair becomes infinities (or NaN at position 0, where it meets a sine of 0);
    # the scale is that of the largest finite rotated magnitude of the block, infinities take the
    # largest code
    rng = np.random.default_rng(109)
    B, Nq, Hq, Hkv, d, page = 2, 21, 4, 2, 64, 16
    c = lsa.LsaPagedKV.empty(B, 9, page, 4, Hkv, d, dtype)
    c.page_table.copy_(torch.tensor([[4, 0, 2, 6], [1, 5, 3, 7]], dtype=torch.int32))
    k, q = _new(rng, B, Nq, Hkv, d), _new(rng, B, Nq, Hq, d)
    inf, nan = float("inf"), float("nan")
    for x in (k, q):
        x[0, 0, 0, 3] = inf                             # position 0
        x[0, 5, 1, 9], x[0, 6, 1, 40], x[0, 7, 1, 2] = inf, -inf, nan
        x[1, 3, 0, 10], x[1, 3, 0, 11], x[1, 3, 0, 42] = inf, -inf, inf
        x[1, 20, 1] = inf                               # a whole row, alone in its block
    v = _new(rng, B, Nq, Hkv, d)
    start = np.array([0, 12], np.int32)
    inv = _freq(d)
    before = _state(c)
    out = lsa.lsa_paged_append(c, k.cuda(), v.cuda(), torch.from_numpy(start).cuda(), q=q.cuda(),
                               inv_freq=torch.from_numpy(inv).cuda(), interleaved=inter)
    c.check()
    want = {n: (None if x is None else x.copy()) for n, x in before.items()}
    with np.errstate(invalid="ignore"):
        wq = plain.append(want, k.float().double().numpy(), v.float().double().numpy(), start, [Nq] * B,
                          inv, inter, q.float().double().numpy())
    g = out.float().cpu().double().numpy()
    assert np.array_equal(np.isnan(g), np.isnan(wq)) and np.array_equal(np.isinf(g), np.isinf(wq))
    assert np.array_equal(np.sign(g)[np.isinf(g)], np.sign(wq)[np.isinf(g)])
    got = _state(c)
    assert np.array_equal(np.isnan(got["K"]), np.isnan(want["K"]))
    if dtype == FP8:
        # no largest magnitude is so near a border of the scale that the rotation's error (2^-21
        # of the pair) passes it; a code may fall on the other side of a half way: one step
        for pg in np.argwhere(want["scales"] > 0)[:, 0]:
            assert np.array_equal(got["scales"][pg], want["scales"][pg])
        top = np.abs(want["K"]) == 448
        assert np.array_equal(got["K"][top], want["K"][top])
        step = plain.half_step(np.nan_to_num(want["K"]))
        near = np.abs(got["K"] - want["K"]) <= 2 * step * 1.0001 + 1e-12
        assert (near | np.isnan(want["K"])).all()
    else:
        assert np.array_equal(np.isinf(got["K"]), np.isinf(want["K"]))
        fin = np.isfinite(want["K"])
        pair = 2.0 ** -21 * 2 * np.nanmax(np.abs(k.float().numpy())[np.isfinite(k.float().numpy())])
        assert (np.abs(got["K"][fin] - want["K"][fin]) <= 2.0 ** -8 * np.abs(want["K"])[fin] + pair).all()


@pytest.mark.parametrize("B,Nq,s", SPLITS)
@pytest.mark.parametrize("q_exp,k_exp,v_exp", [(1, -6, -126), (1, -6, -100), (1, -6, 117),
                                               (110, -115, -64), (-110, 105, 0), (1, -126, -126)])
def test_attention_with_scales_at_the_ends_of_their_range(q_exp, k_exp, v_exp, B, Nq, s):
    # scales from the least normal number to where the values leave bf16's range, the queries such
    # that the logits stay in theirs; factors of up to 2 between blocks
    rng = np.random.default_rng(113)
    Hq, Hkv, d, page, mp = 8, 2, 64, 16, 12
    c = _cache(rng, B, Hkv, d, page, mp, FP8)
    sc = rng.uniform(1.0, 2.0, c.scales.shape)
    sc[:, :, 0] *= 2.0 ** k_exp
    sc[:, :, 1] *= 2.0 ** v_exp
    c.scales.copy_(torch.from_numpy(sc.astype(np.float32)))
    idx, cnt = _rows(rng, B, Nq, mp * page, s, [s, 1, 40, 0, 17])
    Q = torch.from_numpy(rng.standard_normal((B, Nq, Hq, d)) * 2.0 ** q_exp).to(torch.bfloat16)
    O, l = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                              return_lse=True)
    c.check()
    some = np.arange(min(Nq, 12))
    st = _state(c)
    sv = np.repeat(st["scales"], plain.BLOCK, axis=1)
    ro, (ra, floor), rz, rl = plain.attend(
        st["K"] * sv[:, :, 0, :, None], st["V"] * sv[:, :, 1, :, None], st["table"],
        Q[:, some].float().double().numpy(), idx[:, some], cnt[:, some], 1 / np.sqrt(d), sv[:, :, 1])
    dz = 2.0 ** -18 * rz
    # (bf16's subnormals: half of 2^-133)
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 4 * dz)[..., None] * ra + 2.0 ** -31 * floor + 2.0 ** -134
    go = O[:, some].float().cpu().double().numpy()
    assert (np.abs(go - ro) <= tol).all(), np.max(np.abs(go - ro) / tol)
    gl = l[:, some].cpu().double().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (np.abs(gl[~empty] - rl[~empty]) <= (2 * dz + 2.0 ** -19 * (1 + np.abs(rl)))[~empty]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("rows", [1, 10, 11, 15, 16, 24, 25, 26, 35, 36, 52, 53, 71, 75])
def test_attention_of_as_many_rows_as_clusters_fit(dtype, rows):
    # two units to a row: up to and past the clusters of 16, 8, 4 and 2 CTAs that a device holds at
    # once (21, 48, 104, 222 or 31, 71, 142, 296 by the CTAs on an SM), each row whole
    rng = np.random.default_rng(127)
    Hq, Hkv, d, page, mp, s = 6, 2, 128, 32, 4, 2100
    c = _cache(rng, rows, Hkv, d, page, mp, dtype)
    idx, cnt = _rows(rng, rows, 1, mp * page, s, [s, s - 1, s - 33])
    Q = _new(rng, rows, 1, Hq, d).cuda()
    O, l = lsa.lsa_paged_attn(c, Q, torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                              return_lse=True)
    c.check()
    _check_attn(c, Q, idx, cnt, d ** -0.5, O, l)


_FIRST_CALLS = '''
import sys, torch
sys.path.insert(0, sys.argv[1])
import long_context_indexing_b200 as lsa
FP8 = torch.float8_e4m3fn
out = []
with torch.no_grad():
    c = lsa.LsaPagedKV.empty(3, 12, 64, 4, 2, 128, FP8)
    c.page_table.copy_(torch.arange(12, dtype=torch.int32).view(3, 4))
    g0 = torch.Generator().manual_seed(5)
    k = torch.randn(3, 200, 2, 128, generator=g0).bfloat16().cuda()
    q = torch.randn(3, 200, 8, 128, generator=g0).bfloat16().cuda()
    start = torch.zeros(3, dtype=torch.int32, device="cuda")
    idx = torch.randint(0, 200, (3, 1, 150), generator=g0, dtype=torch.int32).cuda()
    cnt = torch.full((3, 1), 150, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qr = lsa.lsa_paged_append(c, k, k, start, q=q)
        O = lsa.lsa_paged_attn(c, q[:, :1].contiguous(), idx, cnt)
    g.replay()
    torch.cuda.synchronize()
    P = lsa.lsa_paged_attn(c, q[:, :1].contiguous(), idx, cnt)
    assert torch.equal(O, P) and O.float().abs().max() > 0
    c.check()
print("same")
'''


def test_first_calls_of_a_process_captured():
    # what a call asks of the device once is asked inside the capture
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS, root], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def test_append_turns_by_large_frequencies_at_far_positions():
    # the angle's product to 2^-31 of a turn for every frequency up to 2^44: against exact
    # fractions of a turn (1 / (2 pi) to 400 bits by Machin's formula)
    from fractions import Fraction

    def arctan_inv(x):
        t = (1 << 420) // x
        s, n, sign = t, 3, -1
        while t:
            t //= x * x
            s, n, sign = s + sign * (t // n), n + 2, -sign
        return s

    inv_2pi = Fraction(1 << 420, 8 * (4 * arctan_inv(5) - arctan_inv(239)))
    rng = np.random.default_rng(131)
    d, page, rot = 64, 1024, 64
    inv = (2.0 ** rng.uniform(-30, 44, rot // 2)).astype(np.float32) * rng.choice([-1, 1], rot // 2)
    inv = inv.astype(np.float32)
    inv[:4] = [2.0 ** 44, -(2.0 ** 44), 0.0, 2.0 ** 44 * (1 - 2.0 ** -24)]
    at = np.array([0, 1, 10485759, 2 ** 31 - 1025], np.int32)
    B = len(at)
    table = torch.full((B, (2 ** 31 - 1) // page), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, at[b] // page] = b
    pages = torch.zeros(B, page, 1, d, dtype=torch.bfloat16, device="cuda")
    c = lsa.LsaPagedKV(pages, pages.clone(), table)
    k = _new(rng, B, 1, 1, d)
    q = _new(rng, B, 1, 2, d)
    out = lsa.lsa_paged_append(c, k.cuda(), k.cuda(), torch.from_numpy(at).cuda(), q=q.cuda(),
                               inv_freq=torch.from_numpy(inv).cuda())
    c.check()
    for b in range(B):
        a = np.array([float((int(at[b]) * Fraction(float(f)) * inv_2pi) % 1) for f in inv]) * 2 * np.pi
        for x, y in ((q[b, 0], out[b, 0]), (k[b, 0], c.k_pages[b, at[b] % page])):
            x, y = x.float().double().numpy(), y.float().cpu().double().numpy()
            u, v = x[:, :rot // 2], x[:, rot // 2:]
            want = np.concatenate([u * np.cos(a) - v * np.sin(a), v * np.cos(a) + u * np.sin(a)], 1)
            pair = np.tile(np.abs(u) + np.abs(v), 2)
            assert (np.abs(y - want) <= 2.0 ** -8 * np.abs(want) + 1.01 * 2.0 ** -21 * pair).all()
