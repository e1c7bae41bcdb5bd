"""The paged cache's entries refuse bad arguments on the host, before any launch,
and the plain binary64 forms that the GPU tests compare with agree with torch."""
import ctypes

import numpy as np
import pytest
import torch

import long_context_indexing_b200 as lsa
import paged_plain as plain

FAKE = 1 << 22


def _kv(**over):
    f = dict(K=FAKE, V=FAKE, scales=FAKE, page_table=FAKE, status=FAKE, B=2, n_pages=10,
             max_pages=5, page=64, Hkv=2, d=128, format=lsa.KV_E4M3)
    f.update(over)
    return lsa.PagedKV(*[f[n] for n, _ in lsa.PagedKV._fields_])


def _append(kv=None, **over):
    a = dict(k=FAKE, ks=256, v=FAKE, vs=256, q=FAKE, qs=1024, q_out=FAKE, Nq=3, Hq=8, start=FAKE,
             n_new=None, inv=FAKE, rot=128, inter=0, stream=None)
    a.update(over)
    return lsa._lib.lsa_paged_append(None if kv == 0 else ctypes.byref(kv or _kv()), *a.values())


def _attn(kv=None, **over):
    a = dict(Q=FAKE, Nq=3, Hq=8, idx=FAKE, cnt=FAKE, s_max=10, scale=0.1, O=FAKE, lse=None,
             stream=None)
    a.update(over)
    return lsa._lib.lsa_paged_attn(None if kv == 0 else ctypes.byref(kv or _kv()), *a.values())


@pytest.mark.parametrize("call", [_append, _attn])
@pytest.mark.parametrize("over,code", [
    (dict(K=None), 1), (dict(V=None), 1), (dict(page_table=None), 1), (dict(status=None), 1),
    (dict(scales=None), 1), (dict(format=2), 1), (dict(B=0), 1), (dict(B=65536), 1),
    (dict(page=48), 7), (dict(page=8), 7), (dict(page=2048), 7), (dict(page=0), 7),
    (dict(n_pages=0), 1), (dict(max_pages=0), 1), (dict(max_pages=1 << 26), 1), (dict(n_pages=1 << 25), 7),
    (dict(d=96), 7), (dict(Hkv=0), 1), (dict(Hkv=3), 1), (dict(K=FAKE + 8), 2),
    (dict(scales=FAKE + 4), 2), (dict(status=FAKE + 4), 2)])
def test_cache_descriptions_refused(call, over, code):
    # (Hkv = 3 with 8 query heads and rows of 256 elements fits neither call)
    assert call(_kv(**over)) == code
    assert lsa._lib.lsa_last_error() != b""


@pytest.mark.parametrize("over,code", [
    (dict(k=None), 1), (dict(v=None), 1), (dict(start=None), 1), (dict(q=None), 1),
    (dict(q_out=None), 1), (dict(Nq=-1), 1), (dict(Nq=1 << 31), 1), (dict(Hq=0), 1),
    (dict(Hq=7), 1), (dict(ks=255), 1), (dict(vs=248), 1), (dict(ks=260), 2), (dict(qs=1016), 1),
    (dict(qs=1032), 1),            # q_out == q with rows apart
    (dict(rot=130), 1), (dict(rot=8), 1), (dict(rot=144), 1), (dict(rot=-16), 1),
    (dict(inv=None), 1), (dict(k=FAKE + 2), 2), (dict(q_out=FAKE + 8), 2), (dict(inv=FAKE + 4), 2)])
def test_append_arguments_refused(over, code):
    assert _append(**over) == code
    assert lsa._lib.lsa_last_error() != b""


@pytest.mark.parametrize("over,code", [
    (dict(Q=None), 1), (dict(idx=None), 1), (dict(cnt=None), 1), (dict(O=None), 1),
    (dict(Nq=-1), 1), (dict(Nq=1 << 30), 7), (dict(s_max=0), 1), (dict(Hq=7), 1),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(Q=FAKE + 8), 2), (dict(lse=FAKE + 4), 2)])
def test_attn_arguments_refused(over, code):
    assert _attn(**over) == code
    assert lsa._lib.lsa_last_error() != b""


def test_null_cache_refused():
    assert _append(0) == 1 and _attn(0) == 1
    assert lsa._lib.lsa_paged_check(None, None) == 1


def test_empty_calls_and_calls_without_gpu():
    assert _append(Nq=0) == 0 and _attn(Nq=0) == 0
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _append() == 4 and _attn() == 4            # LSA_ERR_CUDA, nothing crashes
    assert lsa._lib.lsa_paged_check(ctypes.byref(_kv()), None) == 4


def _index(B=2, dtype=lsa.BF16, T_cap=8192):
    P = lsa.IndexParams(4, 256, 8, 3)
    need = lsa._lib.lsa_index_bytes(B, T_cap, P, dtype)
    h = ctypes.c_void_p()
    assert lsa._lib.lsa_index_init(ctypes.c_void_p(FAKE), need, B, T_cap, P, dtype,
                                   ctypes.byref(h)) == 0
    return h


def _step(h, kv=None, **over):
    S = over.pop("sp", lsa.SelectParams(256, 64, 4))
    a = dict(lat=FAKE, nlk=FAKE, nk=FAKE, nv=FAKE, lq=FAKE, q=FAKE, pos=FAKE, Hq=8, sp=S, inv=FAKE,
             rot=128, inter=0, ws=FAKE, bytes=1 << 40, O=FAKE, stream=None)
    a.update(over)
    return lsa._lib.lsa_decode_step_paged(h, ctypes.byref(kv or _kv()), *a.values())


def test_decode_step_arguments_refused():
    h = _index()
    for over, code in ((dict(lat=None), 1), (dict(nk=None), 1), (dict(q=None), 1), (dict(O=None), 1),
                       (dict(ws=None), 1), (dict(Hq=7), 1), (dict(inv=None), 1), (dict(rot=24), 1),
                       (dict(nv=FAKE + 8), 2), (dict(sp=lsa.SelectParams(256, 2, 4)), 7)):
        assert _step(h, **over) == code, over
    assert _step(h, _kv(B=3)) == 1                          # not the index's sequences
    assert _step(h, _kv(page=24)) == 7
    assert _step(h) == 1                                    # no closed block yet
    assert _step(_index(dtype=lsa.F32)) == 7
    S = lsa.SelectParams(256, 64, 4)
    f = lsa._lib.lsa_decode_paged_workspace_bytes
    n = f(h, ctypes.byref(_kv()), 8, S)
    assert n > 2 * 324 * 4 + 2 * 8 * 128 * 2
    assert f(h, ctypes.byref(_kv(d=96)), 8, S) == 0 and f(h, ctypes.byref(_kv()), 7, S) == 0
    assert f(None, ctypes.byref(_kv()), 8, S) == 0
    assert f(h, ctypes.byref(_kv()), 8, lsa.SelectParams(-1, 64, 4)) == 0


@pytest.mark.parametrize("s_max,code", [(1 << 30, 0), ((1 << 30) + 1, 7), (2 ** 31 - 1, 7)])
def test_rows_whose_tiles_would_pass_32_bits_refused(s_max, code):
    # a tile's places and three steps of 64 tiles of 32 past the row's end must fit 32 bits
    assert (1 << 30) + 4 * 64 * 32 < 2 ** 31
    assert _attn(Nq=0, s_max=s_max) == code          # (no launch either way)
    h = _index()
    f = lsa._lib.lsa_decode_paged_workspace_bytes
    n = f(h, ctypes.byref(_kv()), 8, lsa.SelectParams(s_max - 68, 64, 4))
    assert (n > 0) == (code == 0)
    assert _step(h, sp=lsa.SelectParams(s_max - 68, 64, 4)) == 1
    assert (b"budget+window+sinks" in lsa._lib.lsa_last_error()) == (code != 0)


def test_python_refuses_rows_past_32_bits():
    # a row of 2^32 + 5 positions must not reach the library as one of 5
    import types
    cache = types.SimpleNamespace(B=1, d=64, _index=-1, device=torch.device("cpu"), _addr=0, _ref=None)
    Q = torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)
    idx = torch.zeros(1, dtype=torch.int32).expand(1, 1, 2 ** 32 + 5)
    cnt = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(lsa, "_binding", None)
        m.setattr(lsa, "_current_device", lambda: -1)
        with pytest.raises(ValueError, match="2\\^30"):
            lsa.lsa_paged_attn(cache, Q, idx, cnt)


def _sp(*a):
    return lsa.SelectParams(*a)


@pytest.mark.parametrize("sp", [(0, 0, 0), (2 ** 31 - 1, 1, 0), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1)])
def test_decode_selections_without_a_key_or_past_int_refused(sp):
    # an index of single keys (p = 1) lets the window be 0, so that nothing else refuses them
    P = lsa.IndexParams(1, 256, 8, 3)
    need = lsa._lib.lsa_index_bytes(2, 8192, P, lsa.BF16)
    h = ctypes.c_void_p()
    assert lsa._lib.lsa_index_init(ctypes.c_void_p(FAKE), need, 2, 8192, P, lsa.BF16,
                                   ctypes.byref(h)) == 0
    kv = ctypes.byref(_kv())
    assert lsa._lib.lsa_decode_paged_workspace_bytes(h, kv, 8, _sp(*sp)) == 0
    assert b"budget+window+sinks" in lsa._lib.lsa_last_error()
    assert lsa._lib.lsa_decode_workspace_bytes(h, 8, 2, 128, _sp(*sp)) == 0
    assert _step(h, sp=_sp(*sp)) == 1
    assert b"budget+window+sinks" in lsa._lib.lsa_last_error()
    assert lsa._lib.lsa_decode_step(h, *[FAKE] * 9, 8, 2, 128, _sp(*sp), FAKE, 1 << 40, FAKE, None) == 1
    assert b"budget+window+sinks" in lsa._lib.lsa_last_error()
    # one key is a selection
    assert lsa._lib.lsa_decode_paged_workspace_bytes(h, kv, 8, _sp(0, 0, 1)) > 0
    assert lsa._lib.lsa_decode_workspace_bytes(h, 8, 2, 128, _sp(0, 0, 1)) > 0


def test_binding_is_built_for_this_torch_and_steps_aside():
    # wrong arguments of every kind come back as NotImplemented, for the Python path to name
    b = lsa._binding
    assert b is not None and b.torch_version == torch.__version__
    k = torch.zeros(2, 1, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, 1, 3, dtype=torch.int32)
    kv = _kv(d=64)
    addr = ctypes.addressof(kv)
    for args in ((addr, 0, k, k, i, None, None, None, None, False), (addr, 0, 1, 2, 3, 4, 5, 6, 7, 8),
                 (addr, 0), (0, 0, k, k, i, None, None, None, None, False)):
        if torch.cuda.is_available() or args[0] == 0 or len(args) != 10:
            assert b.append(*args) is NotImplemented
    assert b.attn(addr, 0) is NotImplemented
    with pytest.raises(TypeError):
        b.bind(1)


def test_handle_wants_cuda_tensors_of_one_kind():
    k = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        lsa.LsaPagedKV(k, k, torch.zeros(1, 4, dtype=torch.int32))


def test_decode_step_wants_the_index_on_the_caches_device():
    # the kernels would read the index's memory from another GPU
    import types
    cache = types.SimpleNamespace(B=1, Hkv=2, d=64, _index=0, device=torch.device("cuda", 0))
    index = types.SimpleNamespace(B=1, T_cap=64, buffer=types.SimpleNamespace(
        device=torch.device("cuda", 1)))
    t = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(lsa, "_current_device", lambda: 0)
        with pytest.raises(ValueError, match="different devices"):
            lsa.lsa_decode_step_paged(index, cache, t, t, t, t, t, t, t, 1, 1, 1)


def test_plain_grid_is_torchs_e4m3():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * np.exp2(rng.uniform(-14, 9, 20000)),
                        np.exp2(np.arange(-14, 9)), 1.0625 * np.exp2(np.arange(-14, 8)), [0.0, 448.0]])
    x = x.astype(np.float32).clip(-448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(plain.grid(x).astype(np.float32), want)
    assert plain.grid(np.inf) == 448 and plain.grid(-np.inf) == -448 and np.isnan(plain.grid(np.nan))


def test_plain_scale_and_rotation():
    assert plain.block_scale(0.0) == 2.0 ** -64 and plain.block_scale(448.0) == 1.0
    assert plain.block_scale(np.nextafter(448.0, 500)) == 2.0 and plain.block_scale(3.5) == 2.0 ** -7
    x = np.arange(8.0)
    assert np.allclose(plain.rotate(x, 1, [np.pi / 2, 0.0], False), [-2, 1, 0, 3, 4, 5, 6, 7])
    assert np.allclose(plain.rotate(x, 1, [np.pi / 2, 0.0], True), [-1, 0, 2, 3, 4, 5, 6, 7])


def test_plain_append_and_attend_on_a_worked_case():
    # two tokens into one block: 3.5 sets the scale 2^-7, then 7.0 doubles it; attention
    # over one position returns its value
    st = dict(K=np.zeros((1, 16, 1, 64)), V=np.zeros((1, 16, 1, 64)),
              scales=np.zeros((1, 1, 2, 1)), table=np.zeros((1, 1), np.int32))
    one = np.zeros((1, 1, 1, 64))
    one[..., 0] = 3.5
    plain.append(st, one, one, [0], [1], np.zeros(0), False)
    assert st["scales"][0, 0, 0, 0] == 2.0 ** -7 and st["K"][0, 0, 0, 0] == 448
    plain.append(st, 2 * one, one, [1], [1], np.zeros(0), False)
    assert st["scales"][0, 0, 0, 0] == 2.0 ** -6 and st["scales"][0, 0, 1, 0] == 2.0 ** -7
    assert st["K"][0, 0, 0, 0] == 224 and st["K"][0, 1, 0, 0] == 448
    Kv = st["K"] * st["scales"][0, 0, 0, 0]
    O, _, _, lse = plain.attend(Kv, Kv, st["table"], 2 * one, np.array([[[1, 0]]]), np.array([[1]]), 1.0)
    assert O[0, 0, 0, 0] == 7.0 and lse[0, 0, 0] == 49.0


def test_dependent_kernels_read_nothing_as_unchanging():
    # these kernels start while the one before them still writes what they will read: no load
    # of theirs may go through the read-only path, and their pointers promise nothing that lets
    # the compiler choose it
    import os
    import re
    src = os.path.join(os.path.dirname(lsa.__file__), "csrc")
    for name in ("k_paged_append.cu", "k_paged_attn.cu", "paged.cuh"):
        with open(os.path.join(src, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__ldg|\.global\.nc|__restrict__|__ldlu", code), name


def test_dependent_kernels_wait_before_they_read():
    # every kernel that may start before its predecessor has ended waits for it in its first
    # statements, on every path and in every launch of a call, and none lets a later one start
    # early: what a kernel may see of earlier writes is promised after its own wait only
    import os
    import re
    src = os.path.join(os.path.dirname(lsa.__file__), "csrc")
    for name in ("k_paged_append.cu", "k_paged_attn.cu"):
        with open(os.path.join(src, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert "launch_dependents" not in code and "grid_release" not in code, name
        kernels = code.split("__global__")[1:]
        assert kernels
        for k in kernels:
            head = k[k.index("{"):k.index("grid_dependency();")]
            assert k.count("grid_dependency();") == 1, name
            # declarations and special registers only: no branch, no access to memory
            assert not re.search(r"\bif\b|\bfor\b|->|\ba\.|\bkv\.", head), (name, head)
