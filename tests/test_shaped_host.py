"""Shaped scores, decode weights and eviction without a GPU: the oracle's pins
(brute force, differences) and the refusals of the C ABI and the binding."""
import ctypes
import math

import numpy as np
import pytest
import torch

import exact_io_aware_tmem_b200 as fa
from exact_io_aware_tmem_b200 import _abi
from oracle import attention as oa
from oracle import shaped as osh


@pytest.fixture(scope="module")
def lib():
    from exact_io_aware_tmem_b200 import build
    build.build()
    return _abi.lib()


# ------------------------------------------------------------------ oracle ---

def _rand(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def test_oracle_without_shape_is_the_plain_oracle():
    q, k, v = _rand(0, 9, 4, 8), _rand(1, 9, 2, 8), _rand(2, 9, 2, 8)
    cu = np.array([0, 5, 5, 9])
    r = osh.forward(q, k, v, cu, True, 0.3)
    o, lse = oa.attention_forward(q, k, v, cu, True, 0.3)
    assert np.allclose(r.o, o, atol=1e-13) and np.allclose(r.lse, lse, atol=1e-13)


def test_oracle_brute_force_one_head():
    n, cap, slope, scale = 6, 2.0, 0.4, 0.7
    q, k, v = _rand(3, n, 1, 4), _rand(4, n, 1, 4), _rand(5, n, 1, 4)
    begin, end = [0, 0, 2, 3, 1, 4], [6, 1, 5, 3, 6, 9]
    r = osh.forward(q, k, v, [0, n], False, scale, cap, [slope], begin, end)
    for i in range(n):
        keys = [j for j in range(n) if begin[i] <= j < end[i]]
        z = [cap * math.tanh(scale * float(q[i, 0] @ k[j, 0]) / cap) - slope * abs(i - j)
             for j in keys]
        if not keys:
            assert (r.o[i] == 0).all() and r.lse[0, i] == -np.inf
            continue
        lse = math.log(math.fsum(math.exp(x) for x in z))
        assert abs(r.lse[0, i] - lse) < 1e-12
        assert np.allclose(r.o[i, 0], sum(math.exp(x - lse) * v[j, 0] for x, j in zip(z, keys)))


@pytest.mark.parametrize("causal,cap,alibi", [(True, 1.5, False), (False, 0.0, True),
                                              (True, 3.0, True)])
def test_oracle_gradient_is_the_difference_quotient(causal, cap, alibi):
    n, H, H_kv, D, scale = 5, 4, 2, 3, 0.6
    x = [_rand(10, n, H, D), _rand(11, n, H_kv, D), _rand(12, n, H_kv, D)]
    g = _rand(13, n, H, D)
    slopes = [0.5, 0.1, 0.2, 0.3] if alibi else None
    begin, end = [0, 0, 1, 2, 5], [5, 5, 4, 5, 5]   # the last query sees nothing
    args = ([0, n], causal, scale, cap, slopes, begin, end)
    r = osh.backward(*x, g, *args)
    rng = np.random.default_rng(0)
    for grad, t in zip((r.dq, r.dk, r.dv), range(3)):
        d = rng.standard_normal(x[t].shape)
        h = 1e-6
        val = [float((osh.forward(*[y + s * h * d if u == t else y for u, y in enumerate(x)],
                                  *args).o * g).sum()) for s in (1, -1)]
        assert abs((val[0] - val[1]) / (2 * h) - (grad * d).sum()) < 1e-7
    assert (r.dq[4] == 0).all()


def test_oracle_decode_is_the_forward_of_the_last_tokens():
    n, Q, H, H_kv, D = 11, 3, 4, 2, 8
    q, k, v = _rand(20, n, H, D), _rand(21, n, H_kv, D), _rand(22, n, H_kv, D)
    slopes = [0.5, 0.25, 0.1, 0.05]
    begin = [max(0, i - 3) for i in range(n)]
    r = osh.forward(q, k, v, [0, n], True, 0.5, 2.0, slopes, begin)
    o, lse, _, w = osh.decode(q[-Q:], k, v, [n], q_len=Q, scale=0.5, page_size=n, cap=2.0,
                              slopes=slopes, window=4)
    assert np.allclose(o, r.o[-Q:]) and np.allclose(lse, r.lse.T[-Q:])
    assert np.allclose(w.sum(-1), Q * H / H_kv)
    # A cache whose lost slots nobody sees gives the same through positions.
    kept = np.array([0, 1, 7, 8, 9, 10])
    pos = np.broadcast_to(kept, (1, H_kv, len(kept)))
    o2, lse2, _, _ = osh.decode(q[-1:], k[kept], v[kept], [len(kept)], q_len=1, scale=0.5,
                                page_size=len(kept), cap=2.0, slopes=slopes, window=4,
                                positions=pos)
    assert np.allclose(o2, o[-1:]) and np.allclose(lse2, lse[-1:])


def test_oracle_kept_slots():
    w = np.array([3.0, 1.0, 3.0, np.nan, 3.0, 0.0, -np.inf, 9.0])
    assert osh.kept_slots(w, 8, 3, 0).tolist() == [0, 2, 7]
    assert osh.kept_slots(w, 8, 3, 2).tolist() == [0, 6, 7]
    assert osh.kept_slots(w, 8, 7, 0).tolist() == [0, 1, 2, 4, 5, 6, 7]   # NaN goes first
    assert osh.kept_slots(w, 3, 5, 5).tolist() == [0, 1, 2]
    assert osh.kept_slots(w, 0, 5, 5).tolist() == []


# ---------------------------------------------------------------- refusals ---

P16 = ctypes.c_void_p(256)


def _shape(**kw):
    s = _abi.ScoreShape(50.0, None, None, None)
    for n, x in kw.items():
        setattr(s, n, x)
    return s


def _fwd(lib, shape, **kw):
    a = dict(q=256, k=256, v=256, o=256, lse=256, B=1, H=2, H_kv=2, N=8, D=64,
             dtype=_abi.FA_BF16, causal=0, scale=0.0, cu=None, max_seqlen=0, total=0)
    a.update(kw)
    return lib.fa_fwd_shaped(*a.values(), ctypes.byref(shape), None)


@pytest.mark.parametrize("kw,code", [
    (dict(H=3), _abi.FA_ERR_INVALID_ARG), (dict(D=96), _abi.FA_ERR_UNSUPPORTED),
    (dict(causal=2), _abi.FA_ERR_INVALID_ARG), (dict(q=None), _abi.FA_ERR_INVALID_ARG),
    (dict(v=264), _abi.FA_ERR_INVALID_ARG), (dict(N=-1), _abi.FA_ERR_INVALID_ARG),
    (dict(dtype=_abi.FA_F32, D=129), _abi.FA_ERR_UNSUPPORTED), (dict(B=0), _abi.FA_OK),
    (dict(N=0), _abi.FA_OK)])
def test_fwd_shaped_arguments(lib, kw, code):
    assert _fwd(lib, _shape(), **kw) == code


@pytest.mark.parametrize("cap", [-1.0, float("inf"), float("nan")])
def test_bad_caps_are_refused(lib, cap):
    assert _fwd(lib, _shape(softcap=cap)) == _abi.FA_ERR_INVALID_ARG
    assert _bwd(lib, _shape(softcap=cap)) == _abi.FA_ERR_INVALID_ARG
    assert _decode(lib, _abi.DecodeShape(cap, None, 0, None, None, 0)) == _abi.FA_ERR_INVALID_ARG


@pytest.mark.parametrize("cap,scale", [(2.0 ** 101, 1.0), (2.0 ** -101, 1.0), (1e-40, 0.0)])
def test_caps_out_of_range_are_refused(lib, cap, scale):
    assert _fwd(lib, _shape(softcap=cap), scale=scale) == _abi.FA_ERR_INVALID_ARG
    assert _bwd(lib, _shape(softcap=cap), scale=scale) == _abi.FA_ERR_INVALID_ARG
    assert _decode(lib, _abi.DecodeShape(cap, None, 0, None, None, 0),
                   scale=scale) == _abi.FA_ERR_INVALID_ARG


def _bwd(lib, shape, ws=256, short=0, **kw):
    a = dict(q=256, k=256, v=256, o=256, lse=256, dout=256, dq=256, dk=256, dv=256, B=1, H=2,
             H_kv=2, N=8, D=64, dtype=_abi.FA_BF16, causal=0, scale=0.0, cu=None, max_seqlen=0,
             total=0)
    a.update(kw)
    need = lib.fa_bwd_shaped_workspace_size(a["B"] * a["N"], a["B"], a["H"], a["D"], a["dtype"])
    return lib.fa_bwd_shaped(*a.values(), ctypes.byref(shape), ws, need - short, None)


def test_bwd_shaped_arguments(lib):
    assert _bwd(lib, _shape(), short=1) == _abi.FA_ERR_INVALID_ARG
    assert _bwd(lib, _shape(), ws=128) == _abi.FA_ERR_INVALID_ARG
    assert _bwd(lib, _shape(), dk=None) == _abi.FA_ERR_INVALID_ARG
    assert _bwd(lib, _shape(), dv=264) == _abi.FA_ERR_INVALID_ARG
    assert _bwd(lib, _shape(), N=0) == _abi.FA_OK
    ws = lib.fa_bwd_shaped_workspace_size
    assert ws(-1, 1, 2, 64, _abi.FA_BF16) == 0 and ws(8, -1, 2, 64, _abi.FA_BF16) == 0
    assert ws(1000, 3, 16, 128, _abi.FA_BF16) >= lib.fa_bwd_workspace_size(1000, 16, 128, 0)


def test_key_ranges_arguments(lib):
    def call(prefix=None, window=0, causal=1, B=1, N=8, begin=256, end=256):
        return lib.fa_key_ranges(None, prefix, window, causal, B, N, None, 0, 0, begin, end, None)
    assert call(window=-1) == _abi.FA_ERR_INVALID_ARG
    assert call(prefix=256, causal=0) == _abi.FA_ERR_INVALID_ARG
    assert call(begin=None) == _abi.FA_ERR_INVALID_ARG
    assert call(B=0) == _abi.FA_OK and call(N=0) == _abi.FA_OK


def _decode(lib, shape, **kw):
    a = dict(q=256, k=256, v=256, o=256, lse=256, lens=256, table=None, B=2, q_len=1, H=8, H_kv=2,
             D=128, page=1024, max_blocks=0, rows=2048, max_len=1000, causal=1, scale=-1.0)
    a.update(kw)
    return lib.fa_decode_shaped(*a.values(), None if shape is None else ctypes.byref(shape), None,
                                0, None)


def test_decode_shaped_arguments(lib):
    plain = _abi.DecodeShape(30.0, None, 0, None, None, 0)
    bad, no = _abi.FA_ERR_INVALID_ARG, _abi.FA_ERR_UNSUPPORTED
    assert _decode(lib, None) == bad
    assert _decode(lib, _abi.DecodeShape(0.0, None, -1, None, None, 0)) == bad
    assert _decode(lib, _abi.DecodeShape(0.0, None, 0, None, 256, 999)) == bad   # slots < max_len
    assert _decode(lib, _abi.DecodeShape(0.0, None, 0, 256, None, 999)) == bad
    assert _decode(lib, plain, H=6, H_kv=4) == bad
    assert _decode(lib, plain, D=96) == no
    assert _decode(lib, plain, q_len=9, H=64, H_kv=8) == no       # 72 rows > 64
    assert _decode(lib, plain, page=999) == bad
    assert _decode(lib, plain, table=P16, page=48, max_blocks=64) == no
    assert _decode(lib, plain, q=None) == bad
    assert _decode(lib, plain, B=0) == _abi.FA_OK
    ws = lib.fa_decode_shaped_workspace_size
    assert ws(0, 1, 8, 2, 128, 1000, 1) == 0 and ws(2, 1, 8, 2, 128, -1, 1) == 0
    assert ws(2, 1, 8, 2, 128, 1000, 1) >= ws(2, 1, 8, 2, 128, 1000, 0)


def _evict(lib, **kw):
    big = 1 << 30
    a = dict(k=big, v=2 * big, lens=256, table=None, B=2, H_kv=2, D=128, page=1024, max_blocks=0,
             rows=2048, max_len=1000, weights=256, positions=None, slots=1000, keep=100, recent=10,
             k_out=3 * big, v_out=4 * big, out_table=None, out_page=100, out_blocks=0,
             out_rows=200, seqlens_out=256, weights_out=256, positions_out=256, out_slots=100,
             ws=256, ws_bytes=1 << 20)
    a.update(kw)
    return lib.fa_cache_evict(*a.values(), None)


@pytest.mark.parametrize("kw", [
    dict(keep=0), dict(keep=-3), dict(recent=101), dict(recent=-1), dict(slots=999),
    dict(out_slots=99), dict(out_page=99), dict(out_rows=199), dict(rows=2000), dict(k=None),
    dict(weights=None), dict(weights_out=None), dict(v_out=4 * (1 << 30) + 8), dict(ws=None),
    dict(ws_bytes=10), dict(B=-1), dict(max_len=-1),
    dict(k_out=1 << 30), dict(v_out=(1 << 30) + 1024),          # the cache itself
    dict(k_out=1 << 30, out_table=P16, out_page=64, out_blocks=2, out_rows=2048),
    dict(k_out=4 * (1 << 30) + 1024)])                          # k_out over v_out
def test_evict_refuses(lib, kw):
    assert _evict(lib, **kw) == _abi.FA_ERR_INVALID_ARG


def test_evict_other_statuses(lib):
    assert _evict(lib, D=12) == _abi.FA_ERR_UNSUPPORTED
    assert _evict(lib, D=512) == _abi.FA_ERR_UNSUPPORTED
    assert _evict(lib, out_table=P16, out_page=48, out_blocks=9) == _abi.FA_ERR_UNSUPPORTED
    assert _evict(lib, B=0) == _abi.FA_OK
    assert lib.fa_cache_evict_workspace_size(2, 3, 100) == 2560
    assert lib.fa_cache_evict_workspace_size(0, 3, 100) == 0


def test_binding_refuses_side_tensors_that_do_not_fit():
    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fwd(q, q, q, softcap=30.0)                       # no CUDA tensors
    k = torch.zeros(8, 2, 64, dtype=torch.bfloat16)
    lens = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.decode(k, k, k, lens, q_len=1, max_seqlen_k=4, softcap=30.0, n_split=2)
    with pytest.raises(ValueError):
        fa.decode(k, k, k, lens, q_len=1, max_seqlen_k=4, softcap=30.0)
    with pytest.raises(ValueError):
        fa.evict(k, k, lens, torch.zeros(2, 2, 4), keep=2, max_seqlen_k=4)
    with pytest.raises(ValueError):
        fa.key_ranges()
    with pytest.raises(ValueError):
        fa.key_ranges(doc_ids=torch.zeros(1, 8, dtype=torch.int32))
    with pytest.raises(ValueError):
        fa.key_ranges(8, device="cpu")
