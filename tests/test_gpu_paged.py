"""The paged KV cache on the GPU against binary64 (tests/paged_plain.py).

Tolerances, from the roundings each result passes (eps/2 relative: bf16 2^-8,
fp16 2^-11, e4m3 2^-4 or half its spacing):
  rotation     cos, sin and the two products in fp32: 2^-21 (|x| + |y|) of a pair;
  bf16 pages   one rounding more: 2^-8 of the value;
  8-bit pages  a code is within half the grid's spacing (at the value, over the
               scale) of the rotated value plus the rotation's error; the scale is
               that of a largest magnitude off by the rotation's error at most;
  attention    logits in fp32 over d products: dz = 2^-18 of the largest sum of
               |q k|; weights rounded to fp16 at least, 2^-11, and exp, sum and
               rescaling in fp32: (2^-10 + 4 dz) sum p |v|; output 2^-8 |o| in bf16;
               lse 2 dz + 2^-19 (1 + |lse|).  8-bit pages: the largest weight p sV is
               held at 2^7 or more, so a weight below fp16's normal range is off by
               half of 2^-24 at most, 2^-32 of the largest: 2^-32 max(p sV) sum |codes|,
               twice that for its fp32 exponential.
"""
import numpy as np
import pytest
import torch

import paged_plain as plain

pytestmark = pytest.mark.gpu

lsa = pytest.importorskip("long_context_indexing_b200")

FP8 = torch.float8_e4m3fn


def _freq(rot):
    return (1e6 ** (-np.arange(0, rot, 2) / max(rot, 1))).astype(np.float32)


def _cache(rng, B, Hkv, d, page, max_pages, dtype, spare=2):
    """A cache of random values whose page table is a random permutation."""
    n = B * max_pages + spare
    table = rng.permutation(n)[:B * max_pages].reshape(B, max_pages).astype(np.int32)
    K = torch.from_numpy(rng.standard_normal((n, page, Hkv, d)).astype(np.float32))
    V = torch.from_numpy(rng.standard_normal((n, page, Hkv, d)).astype(np.float32))
    scales = None
    if dtype == FP8:
        K, V = (K * 96).clamp(-448, 448), (V * 96).clamp(-448, 448)
        e = rng.integers(-9, -5, (n, page // 16, 2, Hkv))
        scales = torch.from_numpy(np.exp2(e).astype(np.float32)).cuda()
    return lsa.LsaPagedKV(K.to(dtype).cuda(), V.to(dtype).cuda(), torch.from_numpy(table).cuda(),
                          scales)


def _state(c):
    """The cache as numpy binary64: codes (or bf16 values), scales, table."""
    return dict(K=c.k_pages.float().cpu().double().numpy(),
                V=c.v_pages.float().cpu().double().numpy(),
                scales=None if c.scales is None else c.scales.cpu().double().numpy(),
                table=c.page_table.cpu().numpy())


def _values(st):
    if st["scales"] is None:
        return st["K"], st["V"]
    s = np.repeat(st["scales"], plain.BLOCK, axis=1)          # [n_pages][page][2][Hkv]
    return st["K"] * s[:, :, 0, :, None], st["V"] * s[:, :, 1, :, None]


def _new(rng, B, Nq, H, d):
    """Tokens whose norms spread over a factor of 64, rounded to bf16."""
    x = rng.standard_normal((B, Nq, H, d)) * np.exp2(rng.uniform(-3, 3, (B, Nq, 1, 1)))
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def _pair_sum(x, rot, inter):
    """|x| + |y| of each element's pair."""
    a = np.abs(x).copy()
    r = a[..., :rot].copy()
    if inter:
        o = r.reshape(r.shape[:-1] + (-1, 2))[..., ::-1].reshape(r.shape)
    else:
        o = np.concatenate([r[..., rot // 2:], r[..., :rot // 2]], -1)
    a[..., :rot] = r + o
    return a


def _check_append(c, before, args, got_q=None, q_before=None):
    """The cache after an append against binary64 from its state before."""
    k, v, start, n_new, inv, inter, q = args
    kd, vd = k.float().double().numpy(), v.float().double().numpy()
    qd = None if q is None else q.float().double().numpy()
    want = {n: (None if x is None else x.copy()) for n, x in before.items()}
    wq = plain.append(want, kd, vd, start, n_new, inv, inter, qd)
    got = _state(c)
    rot = 2 * len(inv)
    err = np.zeros_like(want["K"])          # the rotation's error where a key was written
    touched = np.zeros(want["K"].shape[:2], bool)
    page = want["K"].shape[1]
    pair = _pair_sum(kd, rot, inter)
    written = {n: np.full_like(want["K"], np.nan) for n in "KV"}
    for b in range(kd.shape[0]):
        for i in range(min(n_new[b], kd.shape[1])):
            t = int(start[b]) + i
            if start[b] < 0 or t // page >= want["table"].shape[1]:
                continue
            pg = want["table"][b, t // page]
            if pg < 0 or pg >= want["K"].shape[0]:
                continue
            err[pg, t % page] = 2.0 ** -21 * pair[b, i]
            written["K"][pg, t % page] = plain.rotate(kd[b, i], t, inv, inter)
            written["V"][pg, t % page] = vd[b, i]
            touched[pg, t % page] = True
    for j, n in enumerate("KV"):
        e = err if n == "K" else 0.0 * err
        if want["scales"] is None:
            bad = np.abs(got[n] - want[n]) > np.where(touched[..., None, None],
                                                      2.0 ** -8 * np.abs(want[n]) + 1.01 * e, 0.0)
            assert not bad.any(), (n, np.argwhere(bad)[:3])
            continue
        # scales equal, or those of a maximum off by the rotation's error
        gs, ws = got["scales"][:, :, j], want["scales"][:, :, j]
        if n == "V":
            assert np.array_equal(gs, ws)
        else:
            for at in np.argwhere(gs != ws):
                pg, blk, h = at
                w = written[n][pg, blk * 16:(blk + 1) * 16, h]
                m, tol = np.nanmax(np.abs(w)), np.nanmax(err[pg, blk * 16:(blk + 1) * 16, h])
                assert gs[tuple(at)] in (plain.block_scale(m - tol), plain.block_scale(m + tol))
        s = np.repeat(gs, plain.BLOCK, axis=1)[..., None]
        x = written[n]
        step = plain.half_step(np.where(np.isfinite(x), x, 0) / np.where(s > 0, s, 1))
        bad = touched[..., None, None] & np.isfinite(x) & (
            np.abs(got[n] * s - x) > s * step * 1.0001 + 1.01 * e)
        assert not bad.any(), (n, np.argwhere(bad)[:3], got[n][bad][:3], x[bad][:3])
        same = np.broadcast_to(gs == ws, gs.shape)
        rest = ~touched[..., None, None] & np.repeat(same, plain.BLOCK, axis=1)[..., None]
        rest = np.broadcast_to(rest, got[n].shape)
        assert np.array_equal(got[n][rest], want[n][rest], equal_nan=True), n
    if q is not None:
        g = got_q.float().cpu().double().numpy()
        live = ~np.isnan(wq).all(axis=(2, 3))
        tol = 2.0 ** -8 * np.abs(wq) + 1.01 * 2.0 ** -21 * _pair_sum(qd, rot, inter)
        assert (np.abs(g - wq)[live] <= tol[live]).all()
        if q_before is not None:
            old = q_before.float().cpu().double().numpy()
            assert np.array_equal(g[~live], old[~live])


APPEND = [
    # B, Nq, Hq, Hkv, d, page, rot, inter, start
    (1, 1, 8, 1, 128, 16, 128, False, 0),
    (3, 1, 32, 4, 128, 64, 128, False, 37),
    (2, 17, 6, 2, 64, 16, 64, True, 15),
    (1, 100, 24, 3, 128, 32, 64, False, 1),
    (4, 33, 8, 8, 64, 128, 32, True, 63),
    (2, 48, 4, 4, 128, 16, 16, False, 16),
    (1, 5, 16, 16, 64, 1024, 0, False, 9),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,rot,inter,start", APPEND)
def test_append(dtype, B, Nq, Hq, Hkv, d, page, rot, inter, start):
    rng = np.random.default_rng(Nq * 131 + d + rot)
    c = _cache(rng, B, Hkv, d, page, (start + B * 5 + Nq) // page + 1, dtype)
    k, v, q = _new(rng, B, Nq, Hkv, d), _new(rng, B, Nq, Hkv, d), _new(rng, B, Nq, Hq, d)
    st = np.array([start + 5 * b for b in range(B)], np.int32)
    inv = _freq(rot)
    before = _state(c)
    out = lsa.lsa_paged_append(c, k.cuda(), v.cuda(), torch.from_numpy(st).cuda(), q=q.cuda(),
                               inv_freq=torch.from_numpy(inv).cuda() if rot else None,
                               interleaved=inter)
    c.check()
    _check_append(c, before, (k, v, st, [Nq] * B, inv, inter, q), out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_append_padded_batch_from_fused_slices(dtype):
    # unequal lengths with empty and overlong counts; k, v, q sliced from one projection;
    # padding rows hold NaN and are neither read nor written
    rng = np.random.default_rng(3)
    B, Nq, Hq, Hkv, d, page = 5, 40, 8, 2, 128, 32
    c = _cache(rng, B, Hkv, d, page, 4, dtype)
    qkv = _new(rng, B, Nq, Hq + 2 * Hkv, d)
    n_new = np.array([40, 0, 1, 23, 99], np.int32)
    for b in range(B):
        qkv[b, n_new[b]:] = float("nan")
    q, k, v = qkv.split([Hq, Hkv, Hkv], 2)
    dq, dk, dv = qkv.cuda().split([Hq, Hkv, Hkv], 2)
    start = np.array([0, 50, 77, 30, 81], np.int32)
    inv = _freq(128)
    before = _state(c)
    q_out = torch.full((B, Nq, Hq, d), 7.0, dtype=torch.bfloat16, device="cuda")
    q0 = q_out.clone()
    r = lsa.lsa_paged_append(c, dk, dv, torch.from_numpy(start).cuda(),
                             n_new=torch.from_numpy(n_new).cuda(), q=dq, q_out=q_out,
                             inv_freq=torch.from_numpy(inv).cuda())
    assert r is q_out
    c.check()
    _check_append(c, before, (k, v, start, n_new.tolist(), inv, False, q), q_out, q0)


def test_append_token_by_token_grows_scales():
    # one token a call with norms that rise and fall by up to 2^9: every step against
    # binary64 from the step before, among them blocks of zeros, then of tiny values
    rng = np.random.default_rng(11)
    B, Hkv, d, page = 2, 2, 64, 16
    c = lsa.LsaPagedKV.empty(B, 6, page, 3, Hkv, d, FP8)
    c.page_table.copy_(torch.tensor([[4, 0, 2], [1, 5, 3]], dtype=torch.int32))
    inv = _freq(64)
    dinv = torch.from_numpy(inv).cuda()
    for t in range(40):
        size = [0.0, 2.0 ** -30, 2.0 ** rng.uniform(-4, 5), 2.0 ** rng.uniform(-4, 5)][rng.integers(4)]
        k = (_new(rng, B, 1, Hkv, d).float() * size).to(torch.bfloat16)
        v = (_new(rng, B, 1, Hkv, d).float() * size).to(torch.bfloat16)
        st = np.full(B, t, np.int32)
        before = _state(c)
        lsa.lsa_paged_append(c, k.cuda(), v.cuda(), torch.from_numpy(st).cuda(), inv_freq=dinv)
        _check_append(c, before, (k, v, st, [1] * B, inv, False, None))
    c.check()


def test_append_non_finite_values():
    # infinities take the largest code and do not enter the scale; NaN stays NaN
    rng = np.random.default_rng(5)
    c = lsa.LsaPagedKV.empty(1, 1, 16, 1, 1, 64, FP8)
    k, v = _new(rng, 1, 16, 1, 64), _new(rng, 1, 16, 1, 64)
    v[0, 3, 0, 5], v[0, 4, 0, 6], v[0, 5, 0, 7] = float("inf"), float("-inf"), float("nan")
    c.page_table.zero_()
    lsa.lsa_paged_append(c, k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    fin = v.float()[torch.isfinite(v.float())].abs().max().item()
    assert c.scales[0, 0, 1, 0].item() == plain.block_scale(fin)
    got = c.v_pages.float().cpu()[0, :, 0]
    assert got[3, 5] == 448 and got[4, 6] == -448 and torch.isnan(got[5, 7])
    assert torch.isfinite(got).sum() == 16 * 64 - 1


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_append_out_of_range_is_left_out_and_recorded(dtype):
    rng = np.random.default_rng(8)
    B, Nq, Hkv, d, page = 5, 20, 2, 64, 16
    c = _cache(rng, B, Hkv, d, page, 4, dtype)
    table = c.page_table
    table[0, 1], table[1, 1] = -1, 10 ** 6          # no page; a page outside the pool
    start = np.array([0, 10, -3, 2 ** 31 - 10, 55], np.int32)    # 55: runs past the table
    k, v = _new(rng, B, Nq, Hkv, d), _new(rng, B, Nq, Hkv, d)
    before = _state(c)
    lsa.lsa_paged_append(c, k.cuda(), v.cuda(), torch.from_numpy(start).cuda())
    with pytest.raises(lsa.LsaError) as e:
        c.check()
    assert e.value.code == 1
    c.check()                                       # the status was cleared
    _check_append(c, before, (k, v, start, [Nq] * B, _freq(0), False, None))


def test_append_rotates_far_positions_and_in_place():
    # positions up to 2^31 - 1: angles far past what 32 bits hold; q_out is q itself
    rng = np.random.default_rng(9)
    d, page = 128, 1024
    far = np.array([10485759, 2 ** 27 + 1, 2 ** 31 - 1025], np.int32)
    B = len(far)
    table = torch.full((B, (2 ** 31 - 1) // page), -1, dtype=torch.int32, device="cuda")
    for b in range(B):
        table[b, far[b] // page] = b
    pages = torch.zeros(B, page, 1, d, dtype=torch.bfloat16, device="cuda")
    c = lsa.LsaPagedKV(pages, pages.clone(), table)
    k, q = _new(rng, B, 1, 1, d), _new(rng, B, 1, 2, d)
    inv = _freq(128)
    dq = q.cuda()
    out = lsa.lsa_paged_append(c, k.cuda(), k.cuda(), torch.from_numpy(far).cuda(), q=dq, q_out=dq,
                               inv_freq=torch.from_numpy(inv).cuda())
    c.check()
    assert out is dq
    for b in range(B):
        for x, y in ((q[b, 0], dq[b, 0]), (k[b, 0], c.k_pages[b, far[b] % page])):
            want = plain.rotate(x.float().numpy(), far[b], inv, False)
            got = y.float().cpu().double().numpy()
            tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * _pair_sum(x.float().double().numpy(), d, False)
            assert (np.abs(got - want) <= 1.01 * tol).all()


# ---- attention ----------------------------------------------------------------------------------

def _check_attn(c, Q, idx, cnt, scale, O, lse):
    st = _state(c)
    Kv, Vv = _values(st)
    Qd = Q.float().cpu().double().numpy()
    sV = None if st["scales"] is None else np.repeat(st["scales"], plain.BLOCK, axis=1)[:, :, 1]
    ro, ra, rz, rl = plain.attend(Kv, Vv, c.page_table.cpu().numpy(), Qd, idx, cnt, scale, sV)
    ra, floor = ra if sV is not None else (ra, 0.0)
    dz = 2.0 ** -18 * rz
    tol = 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 4 * dz)[..., None] * ra + 2.0 ** -31 * floor + 1e-38
    go = O.float().cpu().double().numpy()
    assert (np.abs(go - ro) <= tol).all(), np.max(np.abs(go - ro) / tol)
    gl = lse.cpu().double().numpy()
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    ok = np.abs(gl - np.where(empty, 0, rl))[~empty] <= \
        (2 * dz + 2.0 ** -19 * (1 + np.abs(rl)))[~empty]
    assert ok.all()


def _rows(rng, B, Nq, T, s_max, counts):
    idx = np.full((B, Nq, s_max), -1, np.int32)
    cnt = np.zeros((B, Nq), np.int32)
    for r in range(B * Nq):
        n = counts[r % len(counts)]
        cnt[r // Nq, r % Nq] = n
        idx[r // Nq, r % Nq, :n] = rng.choice(T, n, replace=n > T)
    return idx, cnt


ATTN = [
    # B, Nq, Hq, Hkv, d, page, max_pages, s_max, counts
    (1, 1, 8, 1, 128, 16, 4, 40, [40]),
    (2, 3, 32, 4, 128, 64, 3, 170, [170, 1, 0, 33, 64, 15]),
    (3, 5, 24, 8, 64, 32, 4, 100, [100, 99, 0, 2, 17]),
    (1, 4, 5, 1, 64, 16, 9, 31, [31, 16, 7, 0]),
    (2, 1, 16, 1, 128, 128, 1, 128, [128, 127]),
    (1, 2, 2, 2, 64, 1024, 1, 700, [700, 513]),
    (4, 1, 28, 4, 128, 16, 40, 640, [640, 0, 639, 333]),
    (1, 1, 32, 4, 128, 64, 80, 5000, [5000]),
    (2, 40, 6, 3, 128, 32, 2, 1, [1, 0]),
    (1, 1, 80, 1, 64, 16, 4, 64, [50]),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,max_pages,s_max,counts", ATTN)
def test_attention(dtype, B, Nq, Hq, Hkv, d, page, max_pages, s_max, counts):
    rng = np.random.default_rng(Hq * 17 + s_max)
    c = _cache(rng, B, Hkv, d, page, max_pages, dtype)
    idx, cnt = _rows(rng, B, Nq, max_pages * page, s_max, counts)
    Q = torch.from_numpy((rng.standard_normal((B, Nq, Hq, d)) * 2).astype(np.float32)).to(torch.bfloat16)
    O, lse = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(),
                                torch.from_numpy(cnt).cuda(), return_lse=True)
    c.check()
    _check_attn(c, Q, idx, cnt, 1 / np.sqrt(d), O, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_attention_never_reads_unlisted_slots(dtype):
    # every slot that no row lists holds NaN, every scale of a block without a listed
    # slot too; indices behind a row's count are garbage
    rng = np.random.default_rng(21)
    B, Nq, Hq, Hkv, d, page, mp, s = 2, 3, 16, 2, 128, 32, 6, 50
    c = _cache(rng, B, Hkv, d, page, mp, dtype)
    idx, cnt = _rows(rng, B, Nq, mp * page, s, [50, 13, 0, 1, 37, 16])
    keep = np.zeros((c.k_pages.shape[0], page), bool)
    table = c.page_table.cpu().numpy()
    for b in range(B):
        for i in range(Nq):
            t = idx[b, i, :cnt[b, i]]
            keep[table[b, t // page], t % page] = True
            idx[b, i, cnt[b, i]:] = rng.integers(-5, 10 ** 9, s - cnt[b, i])
    gone = torch.from_numpy(~keep).cuda()
    for x in (c.k_pages, c.v_pages):
        if dtype == FP8:
            x.view(torch.uint8)[gone] = 0x7F
        else:
            x[gone] = float("nan")
    if dtype == FP8:
        dead = ~keep.reshape(-1, page // 16, 16).any(-1)
        c.scales[torch.from_numpy(dead).cuda()] = float("nan")
    Q = _new(rng, B, Nq, Hq, d)
    O, lse = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(),
                                torch.from_numpy(cnt).cuda(), return_lse=True)
    c.check()
    st = _state(c)
    st["K"], st["V"] = np.nan_to_num(st["K"]), np.nan_to_num(st["V"])
    if st["scales"] is not None:
        st["scales"] = np.nan_to_num(st["scales"])
    Kv, Vv = _values(st)
    ro, ra, rz, rl = plain.attend(Kv, Vv, table, Q.float().double().numpy(), idx, cnt, 1 / np.sqrt(d))
    go = O.float().cpu().double().numpy()
    dz = 2.0 ** -18 * rz
    assert (np.abs(go - ro) <= 2.0 ** -8 * np.abs(ro) + (2.0 ** -10 + 4 * dz)[..., None] * ra).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_attention_skips_and_records_bad_positions(dtype):
    rng = np.random.default_rng(22)
    B, Nq, Hq, Hkv, d, page, mp, s = 2, 2, 8, 2, 64, 16, 8, 90
    c = _cache(rng, B, Hkv, d, page, mp, dtype)
    idx, cnt = _rows(rng, B, Nq, mp * page, s, [90, 90, 60, 3])
    Q = _new(rng, B, Nq, Hq, d)
    idx[0, 0, 5], idx[0, 0, 40], idx[1, 0, 7] = -1, mp * page, 2 ** 31 - 1
    idx[1, 1, :3] = 3                                 # the whole row on a page that is gone
    c.page_table[1, 0] = -1
    c.page_table[0, 2] = c.k_pages.shape[0]
    O, lse = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(),
                                torch.from_numpy(cnt).cuda(), return_lse=True)
    with pytest.raises(lsa.LsaError) as e:
        c.check()
    assert e.value.code == 1
    c.check()
    _check_attn(c, Q, idx, cnt, 1 / np.sqrt(d), O, lse)
    assert (O[1, 1] == 0).all() and torch.isneginf(lse[1, 1]).all()


def test_attention_extreme_logits_and_scales():
    # logits of a few thousand with one key far above the others; V scales 2^20 apart
    # between blocks; K of zeros; any positive scales, powers of two or not
    rng = np.random.default_rng(23)
    B, Nq, Hq, Hkv, d, page, mp, s = 1, 4, 8, 1, 128, 64, 8, 500
    c = _cache(rng, B, Hkv, d, page, mp, FP8)
    sc = np.exp2(rng.uniform(-12, -6, c.scales.shape)).astype(np.float32)
    sc[:, ::2, 1] *= 2.0 ** 20
    c.scales.copy_(torch.from_numpy(sc))
    c.k_pages.view(torch.uint8)[c.page_table[0, 3].item()] = 0
    idx, cnt = _rows(rng, B, Nq, mp * page, s, [500, 400, 300, 2])
    Q = _new(rng, B, Nq, Hq, d).float()
    Q[0, 1] *= 100
    Q[0, 2, ::2] *= 1e4
    Q[0, 2, 1] = 0
    Q[0, 3] *= 1e-6
    Q = Q.to(torch.bfloat16)
    O, lse = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(),
                                torch.from_numpy(cnt).cuda(), return_lse=True)
    c.check()
    _check_attn(c, Q, idx, cnt, 1 / np.sqrt(d), O, lse)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_pages_past_32_bits(dtype):
    # a pool of over 2^32 bytes for each of K and V; the pages in use lie at its end
    page, Hkv, d = 1024, 8, 128
    bytes_page = page * Hkv * d * (1 if dtype == FP8 else 2)
    n = 2 ** 32 // bytes_page + 9
    k = torch.empty(n, page, Hkv, d, dtype=torch.uint8 if dtype == FP8 else dtype, device="cuda")
    v = torch.empty_like(k)
    k, v = (k.view(FP8), v.view(FP8)) if dtype == FP8 else (k, v)
    scales = torch.ones(n, page // 16, 2, Hkv, device="cuda") if dtype == FP8 else None
    table = torch.tensor([[n - 1, n - 3]], dtype=torch.int32, device="cuda")
    c = lsa.LsaPagedKV(k, v, table, scales)
    rng = np.random.default_rng(31)
    N = 2000
    kn, vn = _new(rng, 1, N, Hkv, d), _new(rng, 1, N, Hkv, d)
    lsa.lsa_paged_append(c, kn.cuda(), vn.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    idx = rng.permutation(N)[None, None, :300].astype(np.int32)
    cnt = np.array([[300]], np.int32)
    Q = _new(rng, 1, 1, 16, d)
    O, lse = lsa.lsa_paged_attn(c, Q.cuda(), torch.from_numpy(idx).cuda(),
                                torch.from_numpy(cnt).cuda(), return_lse=True)
    c.check()
    small = lsa.LsaPagedKV(k[-3:].clone(), v[-3:].clone(),
                           torch.tensor([[2, 0]], dtype=torch.int32, device="cuda"),
                           None if scales is None else scales[-3:].clone())
    _check_attn(small, Q, idx, cnt, 1 / np.sqrt(d), O, lse)


def test_streams_graphs_and_two_calls_at_once():
    # the same append and attention eagerly, on a side stream, captured and replayed, and
    # two at once on two streams over two caches give the same bits
    rng = np.random.default_rng(41)
    B, Hq, Hkv, d, page, mp, s = 4, 32, 4, 128, 64, 8, 300
    base = _cache(rng, B, Hkv, d, page, mp, FP8)

    def copy():
        return lsa.LsaPagedKV(base.k_pages.clone(), base.v_pages.clone(), base.page_table.clone(),
                              base.scales.clone())

    k, v, q = (_new(rng, B, 3, h, d).cuda() for h in (Hkv, Hkv, Hq))
    start = torch.tensor([5, 60, 333, 509], dtype=torch.int32, device="cuda")
    inv = torch.from_numpy(_freq(128)).cuda()
    idx, cnt = (torch.from_numpy(x).cuda() for x in _rows(rng, B, 3, mp * page, s, [300, 17, 250]))

    def both(c, stream=None):
        qr = lsa.lsa_paged_append(c, k, v, start, q=q, inv_freq=inv, stream=stream)
        return lsa.lsa_paged_attn(c, qr, idx, cnt, return_lse=True, stream=stream)

    c0 = copy()
    O0, l0 = both(c0)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ca, cb = copy(), copy()
    torch.cuda.synchronize()
    (Oa, la), (Ob, lb) = both(ca, s1), both(cb, s2)
    torch.cuda.synchronize()
    for c, O, l in ((ca, Oa, la), (cb, Ob, lb)):
        assert torch.equal(O, O0) and torch.equal(l, l0)
        assert torch.equal(c.k_pages.view(torch.uint8), c0.k_pages.view(torch.uint8))
        assert torch.equal(c.scales, c0.scales)
    cg = copy()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        Og, lg = both(cg)
    for _ in range(3):
        Og.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Og, O0) and torch.equal(lg, l0)
    cg.check()
    assert torch.equal(cg.v_pages.view(torch.uint8), c0.v_pages.view(torch.uint8))


def test_run_together_with_the_retrieval():
    # chunk by chunk: tokens into pages, latents into the index, the retrieval's selection,
    # attention through the page table; bf16 pages give what lsa_sparse_attn gives over a
    # contiguous cache, 8-bit pages the binary64 attention over their values
    import synth
    w = synth.workload("128k", T=8192, nq=256, M=64, R=512, W=64, S=4)
    inp = synth.prefill_inputs(w, 3, "cpu")
    dev = {n: x.cuda() for n, x in inp.items()}
    span, page = w.p * w.G, 64
    idx = lsa.LsaIndex(1, w.T, w.p, w.G, w.k, w.L, lsa.BF16)
    idx.build(dev["latent_K"], (w.T // span) * span)
    sel, cnt = lsa.lsa_select(idx, dev["latent_Q"], dev["positions"].int(), w.R, w.W, w.S)
    want = lsa.lsa_sparse_attn(dev["Q"], dev["K"], dev["V"], sel, cnt)
    rng = np.random.default_rng(1)
    for dtype in (torch.bfloat16, FP8):
        c = lsa.LsaPagedKV.empty(1, w.T // page, page, w.T // page, w.Hkv, w.d, dtype)
        c.page_table.copy_(torch.from_numpy(rng.permutation(w.T // page).astype(np.int32))[None])
        for t in range(0, w.T, 1000):           # chunks that end inside blocks and pages
            e = min(t + 1000, w.T)
            lsa.lsa_paged_append(c, dev["K"][:, t:e].contiguous(), dev["V"][:, t:e].contiguous(),
                                 torch.tensor([t], dtype=torch.int32, device="cuda"))
        O, lse = lsa.lsa_paged_attn(c, dev["Q"], sel, cnt, return_lse=True)
        c.check()
        if dtype == torch.bfloat16:
            assert (O.float() - want.float()).abs().max() <= 2e-2
        r = np.arange(0, w.nq, 37)
        _check_attn(c, inp["Q"][:, r], sel.cpu().numpy()[:, r], cnt.cpu().numpy()[:, r],
                    1 / np.sqrt(w.d), O[:, r], lse[:, r])


def test_wrong_tensors_are_refused():
    # tensors of wrong shape, type or place are refused before any launch
    c = lsa.LsaPagedKV.empty(2, 4, 16, 2, 2, 64)
    k = torch.zeros(2, 3, 2, 64, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(2, dtype=torch.int32, device="cuda")
    n0 = lsa.kernel_launches()
    for bad in (dict(k=k[:1]), dict(k=k.float()), dict(k=k.cpu()), dict(k=k[..., :32]),
                dict(v=k[:, :2]), dict(v=k.transpose(1, 2)), dict(start=st.long()),
                dict(start=st[:1]), dict(n_new=st[:1]), dict(inv_freq=st),
                dict(inv_freq=torch.zeros(5, device="cuda")), dict(q_out=k),
                dict(q=k[:, :, :1]), dict(k=k[:, :, :1])):
        args = dict(k=k, v=k, start=st)
        args.update(bad)
        with pytest.raises((ValueError, TypeError, lsa.LsaError)):
            lsa.lsa_paged_append(c, args.pop("k"), args.pop("v"), args.pop("start"), **args)
    Q = torch.zeros(2, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    idx = torch.zeros(2, 3, 5, dtype=torch.int32, device="cuda")
    cnt = torch.ones(2, 3, dtype=torch.int32, device="cuda")
    for bad in (dict(Q=Q[:1]), dict(Q=Q.float()), dict(Q=Q[:, :, :3]), dict(indices=idx.long()),
                dict(indices=idx[:, :2]), dict(counts=cnt[:1]), dict(out=Q.float()),
                dict(Q=Q.transpose(1, 2)), dict(scale=0.0), dict(scale=float("nan"))):
        args = dict(Q=Q, indices=idx, counts=cnt)
        args.update(bad)
        with pytest.raises((ValueError, TypeError, lsa.LsaError)):
            lsa.lsa_paged_attn(c, args.pop("Q"), args.pop("indices"), args.pop("counts"), **args)
    assert lsa.kernel_launches() == n0
    # empty calls are allowed and launch nothing
    lsa.lsa_paged_append(c, k[:, :0], k[:, :0], st)
    assert lsa.lsa_paged_attn(c, Q[:, :0].contiguous(), idx[:, :0].contiguous(),
                              cnt[:, :0].contiguous()).shape == (2, 0, 4, 64)
    assert lsa.kernel_launches() == n0


@pytest.mark.parametrize("dtype,Hq,Hkv,d", [(torch.bfloat16, 32, 4, 128), (FP8, 12, 4, 64),
                                            (FP8, 32, 4, 128)])
def test_decode_steps_over_pages(dtype, Hq, Hkv, d):
    # every step: the selection is lsa_decode_step's over the same latents; the appended
    # token and the attention over the selection are those of binary64
    import synth
    w = synth.workload("decode", T=4096, B=3, M=64, G=64, k=4, L=3, R=600, W=8, S=4, steps=20,
                       Hq=Hq, Hkv=Hkv, d=d, dtype="bf16")
    inp = synth.decode_inputs(w, 13, "cpu")
    page, t_cap = 32, w.T + 20 + w.p * w.G
    rng = np.random.default_rng(7)
    n_pages = w.B * ((t_cap + page - 1) // page)
    c = lsa.LsaPagedKV.empty(w.B, n_pages + 1, page, n_pages // w.B, Hkv, d, dtype)
    c.page_table.copy_(torch.from_numpy(rng.permutation(n_pages).reshape(w.B, -1).astype(np.int32)))
    inv = _freq(d)
    dinv = torch.from_numpy(inv).cuda()
    lat = torch.zeros(w.B, t_cap, 64, dtype=torch.bfloat16, device="cuda")
    lat[:, :w.T] = inp["latent_K"][:, :w.T].cuda()
    lsa.lsa_paged_append(c, inp["K"][:, :w.T].cuda(), inp["V"][:, :w.T].cuda(),
                         torch.zeros(w.B, dtype=torch.int32, device="cuda"), inv_freq=dinv)
    idx = lsa.LsaIndex(w.B, t_cap, w.p, w.G, w.k, w.L, lsa.BF16)
    idx.build(lat, w.T)
    # the contiguous path beside it, for the selections
    lat2 = lat.clone()
    idx2 = lsa.LsaIndex(w.B, t_cap, w.p, w.G, w.k, w.L, lsa.BF16)
    idx2.build(lat2, w.T)
    heads = (8, 4) if Hq == 12 else (Hq, Hkv)
    K2 = torch.zeros(w.B, t_cap, heads[1], d, dtype=torch.bfloat16, device="cuda")
    V2 = torch.zeros_like(K2)
    ws = torch.empty(lsa.lsa_decode_paged_workspace_bytes(idx, c, Hq, w.R, w.W, w.S),
                     dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(lsa.lsa_decode_workspace_bytes(idx2, *heads, d, w.R, w.W, w.S),
                      dtype=torch.uint8, device="cuda")
    for t in range(12):
        pos = torch.full((w.B,), w.T + t, dtype=torch.int32, device="cuda")
        new = [inp[n][t].contiguous().cuda() for n in ("new_latent_k", "new_k", "new_v", "latent_q", "q")]
        before = _state(c)
        O = lsa.lsa_decode_step_paged(idx, c, lat, *new, pos, w.R, w.W, w.S, inv_freq=dinv,
                                      workspace=ws)
        sel, cnt = lsa.decode_selection_views(ws, w.B, w.s_max)
        lsa.lsa_decode_step(idx2, lat2, K2, V2, new[0], new[1][:, :heads[1]].contiguous(),
                            new[2][:, :heads[1]].contiguous(), new[3],
                            new[4][:, :heads[0]].contiguous(), pos, w.R, w.W, w.S, workspace=ws2)
        sel2, cnt2 = lsa.decode_selection_views(ws2, w.B, w.s_max)
        assert torch.equal(cnt, cnt2) and torch.equal(sel, sel2) and torch.equal(lat, lat2)
        k, v, q = (new[i].cpu()[:, None] for i in (1, 2, 4))
        _check_append(c, before, (k, v, pos.cpu().numpy(), [1] * w.B, inv, False, None))
        # the queries as the step rotates them
        qr = torch.empty_like(q.cuda())
        spare = lsa.LsaPagedKV(c.k_pages.clone(), c.v_pages.clone(), c.page_table,
                               None if c.scales is None else c.scales.clone())
        lsa.lsa_paged_append(spare, k.cuda(), v.cuda(), pos, q=q.cuda(), q_out=qr, inv_freq=dinv)
        O2, lse = lsa.lsa_paged_attn(c, qr, sel[:, None].contiguous(), cnt[:, None].contiguous(),
                                     return_lse=True)
        assert torch.equal(O, O2[:, 0])
        _check_attn(c, qr, sel[:, None].cpu().numpy(), cnt[:, None].cpu().numpy(), 1 / np.sqrt(d),
                    O[:, None], lse)
    idx.check()
    c.check()


def test_decode_step_captured_and_replayed():
    # one captured step replayed with the position and the inputs changed in place gives
    # what eager steps give
    import synth
    w = synth.workload("decode", T=2048, B=2, M=32, G=64, k=4, L=3, R=300, W=16, S=4, steps=8,
                       Hq=8, Hkv=2, d=64, dtype="bf16")
    inp = synth.decode_inputs(w, 17, "cpu")
    page, t_cap = 16, w.T + 8 + w.p * w.G
    dinv = torch.from_numpy(_freq(64)).cuda()

    def setup():
        mp = (t_cap + page - 1) // page
        c = lsa.LsaPagedKV.empty(w.B, w.B * mp, page, mp, w.Hkv, w.d, FP8)
        c.page_table.copy_(torch.arange(w.B * mp, dtype=torch.int32).view(w.B, mp))
        lat = torch.zeros(w.B, t_cap, 64, dtype=torch.bfloat16, device="cuda")
        lat[:, :w.T] = inp["latent_K"][:, :w.T].cuda()
        lsa.lsa_paged_append(c, inp["K"][:, :w.T].cuda(), inp["V"][:, :w.T].cuda(),
                             torch.zeros(w.B, dtype=torch.int32, device="cuda"), inv_freq=dinv)
        idx = lsa.LsaIndex(w.B, t_cap, w.p, w.G, w.k, w.L, lsa.BF16)
        idx.build(lat, w.T)
        ws = torch.empty(lsa.lsa_decode_paged_workspace_bytes(idx, c, w.Hq, w.R, w.W, w.S),
                         dtype=torch.uint8, device="cuda")
        return c, lat, idx, ws

    names = ("new_latent_k", "new_k", "new_v", "latent_q", "q")
    want = []
    c, lat, idx, ws = setup()
    for t in range(6):
        pos = torch.full((w.B,), w.T + t, dtype=torch.int32, device="cuda")
        want.append(lsa.lsa_decode_step_paged(idx, c, lat, *[inp[n][t].contiguous().cuda() for n in names],
                                              pos, w.R, w.W, w.S, inv_freq=dinv, workspace=ws).clone())
    c, lat, idx, ws = setup()
    x = [inp[n][0].contiguous().cuda() for n in names]
    pos = torch.full((w.B,), w.T, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x[4])
    # one eager step first: the same token again, so that the capture finds the index ready
    lsa.lsa_decode_step_paged(idx, c, lat, *x, pos, w.R, w.W, w.S, inv_freq=dinv, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        lsa.lsa_decode_step_paged(idx, c, lat, *x, pos, w.R, w.W, w.S, inv_freq=dinv, workspace=ws,
                                  out=out)
    for t in range(6):
        for a, n in zip(x, names):
            a.copy_(inp[n][t])
        pos.fill_(w.T + t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[t]), t
    c.check()
    idx.check()


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
def test_compiled_binding_and_python_path_agree(dtype, monkeypatch):
    # the same bits through the compiled binding and through the Python path, with slices,
    # padding, given and new outputs
    rng = np.random.default_rng(51)
    B, Nq, Hq, Hkv, d, page, mp = 3, 9, 12, 4, 64, 16, 6
    base = _cache(rng, B, Hkv, d, page, mp, dtype)
    q, k, v = _new(rng, B, Nq, Hq + 2 * Hkv, d).cuda().split([Hq, Hkv, Hkv], 2)
    start = torch.tensor([3, 40, 80], dtype=torch.int32, device="cuda")
    n_new = torch.tensor([9, 4, 0], dtype=torch.int32, device="cuda")
    inv = torch.from_numpy(_freq(32)).cuda()
    idx, cnt = (torch.from_numpy(x).cuda() for x in _rows(rng, B, Nq, mp * page, 50, [50, 0, 7]))
    assert lsa._binding is not None
    got = []
    for path in range(2):
        if path:
            monkeypatch.setattr(lsa, "_binding", None)
        c = lsa.LsaPagedKV(base.k_pages.clone(), base.v_pages.clone(), base.page_table,
                           None if base.scales is None else base.scales.clone())
        qr = lsa.lsa_paged_append(c, k, v, start, q=q, inv_freq=inv, interleaved=True)
        given = torch.zeros_like(qr)
        assert lsa.lsa_paged_append(c, k, v, start, n_new=n_new, q=q, q_out=given) is given
        assert lsa.lsa_paged_append(c, k, v, start) is None
        O, lse = lsa.lsa_paged_attn(c, qr, idx, cnt, scale=0.3, return_lse=True)
        P = torch.zeros_like(O)
        assert lsa.lsa_paged_attn(c, qr, idx, cnt, out=P) is P
        one = lsa.lsa_paged_attn(c, qr, idx, cnt)
        c.check()
        got.append([qr, given, O, lse, P, one, c.k_pages.view(torch.uint8), c.v_pages.view(torch.uint8)]
                   + ([] if c.scales is None else [c.scales]))
        with pytest.raises(lsa.LsaError) as e:                  # refused by the C entry
            lsa.lsa_paged_attn(c, qr, idx, cnt, scale=-1.0)
        assert e.value.code == 1
    for x, y in zip(*got):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


def test_calls_in_a_row_wait_for_each_other():
    # a long chain without a wait in between: each step appends what the attention before it
    # wrote, among torch's own kernels; the same as with a wait after every call
    rng = np.random.default_rng(61)
    B, Hq, Hkv, d, page, mp = 6, 16, 4, 128, 16, 20
    base = _cache(rng, B, Hkv, d, page, mp, FP8)
    x0 = _new(rng, B, 1, Hq, d).cuda()
    inv = torch.from_numpy(_freq(128)).cuda()
    idx, cnt = (torch.from_numpy(x).cuda() for x in _rows(rng, B, 1, mp * page, 300, [300, 40, 0, 299]))

    def chain(wait):
        c = lsa.LsaPagedKV(base.k_pages.clone(), base.v_pages.clone(), base.page_table,
                           base.scales.clone())
        x, pos = x0.clone(), torch.arange(B, dtype=torch.int32, device="cuda") * 3
        out = []
        for step in range(60):
            qr = lsa.lsa_paged_append(c, x[:, :, :Hkv], x[:, :, Hkv:2 * Hkv], pos, q=x, inv_freq=inv)
            if wait:
                torch.cuda.synchronize()
            x = lsa.lsa_paged_attn(c, qr, idx, cnt)
            if step % 3 == 0:
                x = (x * 1.5 + x0).clamp_(-8, 8)
            pos += 1
            if wait:
                torch.cuda.synchronize()
            out.append(x)
        torch.cuda.synchronize()
        return torch.stack(out), c.k_pages.view(torch.uint8)

    a, ka = chain(True)
    for _ in range(3):
        b, kb = chain(False)
        assert torch.equal(a, b) and torch.equal(ka, kb)


def test_calls_wait_for_other_streams_copies_and_fills():
    # inputs that a slow side stream, a copy and a fill have just written, joined by events,
    # eagerly and as branches of a captured graph: the same as with a wait after everything
    rng = np.random.default_rng(67)
    B, Hq, Hkv, d, page, mp = 5, 16, 4, 128, 32, 12
    base = _cache(rng, B, Hkv, d, page, mp, FP8)
    k0, v0, q0 = (_new(rng, B, 2, h, d).cuda() for h in (Hkv, Hkv, Hq))
    inv = torch.from_numpy(_freq(128)).cuda()
    idx0, cnt0 = (torch.from_numpy(x).cuda() for x in _rows(rng, B, 2, mp * page, 90, [90, 0, 33]))
    side = torch.cuda.Stream()
    main = torch.cuda.Stream()

    def step(c, b, sync):
        here = torch.cuda.current_stream()
        wait = torch.cuda.synchronize if sync else (lambda: None)
        b["start"].fill_(7)                             # a fill straight before
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            b["k"].copy_(k0)
            b["v"].copy_(v0 * 2)
        b["q"].copy_(q0)                                # beside the branch
        wait()
        here.wait_stream(side)
        qr = lsa.lsa_paged_append(c, b["k"], b["v"], b["start"], q=b["q"], inv_freq=inv)
        wait()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            b["idx"].copy_(idx0)
        b["cnt"].copy_(cnt0)
        here.wait_stream(side)
        wait()
        O, l = lsa.lsa_paged_attn(c, qr, b["idx"], b["cnt"], return_lse=True)
        wait()
        b["k"].zero_(), b["q"].zero_(), b["idx"].fill_(-1), b["cnt"].zero_()
        return O, l

    def fresh():
        c = lsa.LsaPagedKV(base.k_pages.clone(), base.v_pages.clone(), base.page_table,
                           base.scales.clone())
        b = dict(k=torch.zeros_like(k0), v=torch.zeros_like(v0), q=torch.zeros_like(q0),
                 idx=torch.full_like(idx0, -1), cnt=torch.zeros_like(cnt0),
                 start=torch.zeros(B, dtype=torch.int32, device="cuda"))
        torch.cuda.synchronize()
        return c, b

    with torch.cuda.stream(main):
        c0, b0 = fresh()
        O0, l0 = step(c0, b0, True)
        c1, b1 = fresh()
        for _ in range(4):
            O, l = step(c1, b1, False)
            torch.cuda.synchronize()
            assert torch.equal(O, O0) and torch.equal(l, l0)
    c2, b2 = fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=main):
        Og, lg = step(c2, b2, False)
    for _ in range(4):
        Og.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(Og, O0) and torch.equal(lg, l0)
    for c in (c1, c2):
        c.check()
        assert torch.equal(c.k_pages.view(torch.uint8), c0.k_pages.view(torch.uint8))
        assert torch.equal(c.v_pages.view(torch.uint8), c0.v_pages.view(torch.uint8))


def test_attention_of_a_position_listed_many_times():
    # every listing counts: a position listed n times weighs n times, within a tile and across
    # the tiles, warps and CTAs of a row
    rng = np.random.default_rng(71)
    for dtype in (torch.bfloat16, FP8):
        c = _cache(rng, 1, 2, 128, 32, 4, dtype)
        Q = _new(rng, 1, 3, 10, 128).cuda()
        idx = np.full((1, 3, 2000), -1, np.int32)
        idx[0, 0] = 5                                   # one position only
        idx[0, 1] = rng.choice([3, 64, 127], 2000)
        idx[0, 2, ::2] = 9
        idx[0, 2, 1::2] = np.arange(1000) % 128
        cnt = np.full((1, 3), 2000, np.int32)
        O, l = lsa.lsa_paged_attn(c, Q, torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                                  return_lse=True)
        c.check()
        _check_attn(c, Q, idx, cnt, 128 ** -0.5, O, l)


@pytest.mark.parametrize("dtype,B,Nq,Hq,Hkv,d", [(torch.bfloat16, 1, 225, 6, 2, 128),
                                                 (FP8, 3, 50, 4, 4, 128), (FP8, 203, 1, 9, 3, 64),
                                                 (torch.bfloat16, 1, 70, 80, 1, 64),
                                                 (torch.bfloat16, 90, 10, 2, 1, 128)])
def test_attention_in_two_launches(dtype, B, Nq, Hq, Hkv, d):
    # a little more than one or two waves of units: the last ones run in a launch of their own
    rng = np.random.default_rng(73)
    page, mp, s = 16, 6, 1030
    c = _cache(rng, B, Hkv, d, page, mp, dtype)
    Q = _new(rng, B, Nq, Hq, d).cuda()
    idx, cnt = _rows(rng, B, Nq, mp * page, s, [1030, 1, 0, 700, 1029, 513, 96])
    before = lsa.kernel_launches()
    O, l = lsa.lsa_paged_attn(c, Q, torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda(),
                              return_lse=True)
    assert lsa.kernel_launches() == before + 2
    c.check()
    _check_attn(c, Q, idx, cnt, d ** -0.5, O, l)


def test_two_launches_are_waited_for_and_wait():
    # attention in two launches between calls that write what it reads and read what it writes,
    # eagerly and captured: the same as with a wait after every call
    rng = np.random.default_rng(79)
    B, Nq, Hq, Hkv, d, page, mp, s = 1, 150, 8, 4, 128, 32, 24, 1100
    base = _cache(rng, B, Hkv, d, page, mp, FP8)
    x0 = _new(rng, B, Nq, Hq, d).cuda()
    inv = torch.from_numpy(_freq(128)).cuda()
    cnt = np.full((B, Nq), s, np.int32)
    idx = rng.integers(0, mp * page, (B, Nq, s)).astype(np.int32)
    # the first launch's rows long, the last ones' short: the second launch ends early
    cnt[:, 148:] = 3
    idx, cnt = torch.from_numpy(idx).cuda(), torch.from_numpy(cnt).cuda()
    pos = torch.tensor([1], dtype=torch.int32, device="cuda")

    def chain(c, wait, steps):
        x, out = x0.clone(), []
        for step in range(steps):
            qr = lsa.lsa_paged_append(c, x[:, :, :Hkv], x[:, :, Hkv:], pos + step, q=x,
                                      inv_freq=inv)
            if wait:
                torch.cuda.synchronize()
            x = lsa.lsa_paged_attn(c, qr, idx, cnt)
            if wait:
                torch.cuda.synchronize()
            if step % 3 == 1:
                x = (x * 1.5 + x0).clamp_(-8, 8)
            if step % 4 == 2:
                qr.zero_()                              # (its launches have read it)
                x = lsa.lsa_paged_attn(c, x, idx, cnt)
            if wait:
                torch.cuda.synchronize()
            out.append(x)
        return torch.stack(out)

    def copy():
        return lsa.LsaPagedKV(base.k_pages.clone(), base.v_pages.clone(), base.page_table,
                              base.scales.clone())

    ca = copy()
    a = chain(ca, True, 20)
    for stream in (torch.cuda.current_stream(), torch.cuda.Stream()):
        cb = copy()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            b = chain(cb, False, 20)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
        assert torch.equal(ca.k_pages.view(torch.uint8), cb.k_pages.view(torch.uint8))
    cg, g = copy(), torch.cuda.CUDAGraph()
    k, v, sc = (t.clone() for t in (cg.k_pages.view(torch.uint8), cg.v_pages.view(torch.uint8),
                                    cg.scales))
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = chain(cg, False, 20)
    for _ in range(3):
        cg.k_pages.view(torch.uint8).copy_(k)
        cg.v_pages.view(torch.uint8).copy_(v)
        cg.scales.copy_(sc)
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, FP8])
@pytest.mark.parametrize("B,Nq,Hq,Hkv,d,page,rot,inter,start", [
    (1, 100, 40, 4, 128, 32, 128, False, 11),     # five parts of the queries
    (2, 17, 21, 3, 64, 16, 32, True, 15),         # two parts, an odd number of heads
    (1, 3, 70, 1, 128, 64, 64, False, 62),        # three parts of a few tokens
    (18, 60, 63, 1, 128, 16, 128, False, 5),      # fewer parts than loads in flight would make
    (40, 50, 24, 2, 128, 32, 128, True, 3),       # one part
    (300, 20, 5, 1, 64, 16, 64, False, 0),        # keys, values and queries in one CTA
])
def test_append_query_parts(dtype, B, Nq, Hq, Hkv, d, page, rot, inter, start):
    test_append(dtype, B, Nq, Hq, Hkv, d, page, rot, inter, start)
