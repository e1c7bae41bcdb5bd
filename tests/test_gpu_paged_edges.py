"""The paged cache's calls at their edges: rows that nothing writes, infinities and NaN, scales at the
ends of their range.  References and tolerances are those of test_gpu_paged.py."""
import numpy as np
import pytest
import torch

import paged_plain as plain
from test_gpu_paged import FP8, _cache, _check_append, _check_attn, _freq, _new, _rows, _state, lsa

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
