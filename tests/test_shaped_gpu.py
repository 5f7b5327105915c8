"""GPU parity of attention with shaped scores (fwd, bwd, key_ranges), of its decode
with accumulated weights, and of cache eviction, against the float64 oracle.

Tolerances, element by element, from the roundings that the kernels make. A value
rounded to bf16 is off by at most 2^-8 of itself. With e the largest error of a
score z in fp32 (the D products' sums, the cap, the base-2 exponent's rounding) plus
1e-4 for the exponentials' own error (7.5e-5 at most):
  O    P rounded to bf16, O rounded:          (2^-8 + 2e) P|V| + 2^-8 |O|
       In the forward's masked tiles the P that are summed are the rounded ones: with P_j
       (1 + d_j), |d_j| <= 2^-8, O = sum (P + P d) V / sum (P + P d) is off by sum P d (V -
       O) / (1 + sum P d) with P summing to 1, at most 2^-8 / (1 - 2^-8) (P|V| + |O|)
       < 2^-8 (1 + 2^-7) (P|V| + |O|).
  LSE                                         e
  dV   as O:                                  (2^-8 + 2e) P^T|dO| + 2^-8 |dV|
  dQ   P (once more for dS) and dS rounded, D_i = sum P dP in fp32, dQ rounded:
       (2^-7 + 4e) scale |dX||K| + (2^-8 + 2e) (what D_i moves) + 2^-8 |dQ|;  dK alike.
       Under a cap 1 - t^2 is formed from a t = tanh that fp32 gives to 2^-22 (a few
       steps of 2^-24, |t| <= 1), and is off by 2 t 2^-22 + 2^-24 < 2^-20 however small
       it is: 2^-20 scale |dZ||K| more.
       P (1 - t^2) 2^14 is held as fp16 for dX: its step below 2^-14 is 2^-24, so P (1 - t^2)
       is off by up to 2^-25 2^-14 = 2^-39 however small it is: 2^-39 scale |dO V^T - D||K| more
float32: the same without the bf16 terms, e without the 1e-4, and 2^-24 a term summed.
"""
import numpy as np
import pytest
import torch

import exact_io_aware_tmem_b200 as fa
from exact_io_aware_tmem_b200.workloads import decode_case, random_case
from oracle import shaped as osh
from tests._util import f64

pytestmark = pytest.mark.gpu

HALF = 2.0 ** -8      # half a bf16 step, relative
# A term below the smallest normal fp32 number (2^-126) has no relative precision: it is
# off by up to 2^-126, times a factor below 2^7 (|v|, |dO|, |k|, scale), summed over at
# most 2^12 terms: 2^-107 < 1e-32.
TINY = 1e-32


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_tmem_b200 import build
    build.build()


def clean():
    st, where = fa.check_device_error()
    assert st == 0, f"device error {st} at {where:#x}"


def score_error(q, k, scale, cap, slopes, n, dtype):
    """Largest error of a score in fp32, plus the exponentials' (see above)."""
    H, H_kv = q.shape[1], k.shape[1]
    dot = np.sqrt((f64(q) ** 2).sum(-1).max() * (f64(k) ** 2).sum(-1).max())   # >= sum |q||k|
    z = min(scale * dot, cap) if cap else scale * dot
    z += 0.0 if slopes is None else float(slopes.max()) * n
    e = q.shape[2] * 2.0 ** -24 * scale * dot + 2.0 ** -21 * (2 + z + cap)
    return e + (1e-4 if dtype == "bf16" else n * 2.0 ** -24)


def inside(name, got, ref, tol):
    got, ref = np.asarray(got), np.asarray(ref)
    assert np.array_equal(np.isneginf(got), np.isneginf(ref)), f"{name}: -inf rows differ"
    fin = ~np.isneginf(ref)
    assert np.isfinite(got[fin]).all(), f"{name}: not finite"
    over = np.abs(got[fin] - ref[fin]) - (tol if np.isscalar(tol) else tol[fin]) - TINY
    assert over.size == 0 or over.max() <= 0, f"{name}: {over.max()} outside its bound"


def ranges_of(mask, lengths, rng):
    """(begin, end) of the tokens for a kind of mask, or (None, None)."""
    if mask == "none":
        return None, None
    begin, end = [], []
    for n in lengths:
        i = np.arange(n)
        if mask == "docs":
            cuts = np.unique(np.concatenate([[0], rng.integers(0, n + 1, 4), [n]]))
            d = np.searchsorted(cuts, i, side="right")
            begin.append(cuts[d - 1] if n else i)
            end.append(cuts[np.minimum(d, len(cuts) - 1)] if n else i)
        elif mask == "prefix":
            begin.append(0 * i)
            end.append(np.maximum(i + 1, int(rng.integers(0, n + 1))))
        elif mask == "window":
            begin.append(np.maximum(0, i - int(rng.integers(0, max(1, n // 2)))))
            end.append(i + 1)
        else:   # anything: empty rows, entries outside the sequence
            begin.append(rng.integers(-5, n + 5, n))
            end.append(rng.integers(-5, n + 9, n))
    return (np.concatenate(begin).astype(np.int32), np.concatenate(end).astype(np.int32))


def run_case(seed, dtype, lengths, H, H_kv, D, varlen, causal, cap, alibi, mask, std=1.0,
             backward=True, scale=None):
    inp = random_case(seed, dtype=dtype, lengths=lengths, H=H, H_kv=H_kv, D=D, varlen=varlen,
                      std=std)
    B, N = len(lengths), max(lengths)
    begin, end = ranges_of(mask, lengths, np.random.default_rng(seed))
    slopes = torch.tensor([0.6 * 0.7 ** h for h in range(H)]) if alibi else None
    scale = D ** -0.5 if scale is None else scale
    T = sum(lengths)

    def dev(t):
        t = t.cuda()
        return t if varlen else t.view(B, N, *t.shape[1:]).contiguous()
    q, k, v, do = dev(inp.q), dev(inp.k), dev(inp.v), dev(inp.do)
    kw = dict(causal=causal, scale=scale, softcap=cap or None,
              alibi_slopes=None if slopes is None else slopes.cuda(),
              key_begin=None if begin is None else dev(torch.from_numpy(begin)),
              key_end=None if end is None else dev(torch.from_numpy(end)))
    if varlen:
        kw.update(cu_seqlens=inp.cu_seqlens.cuda(), max_seqlen=N)
    o, lse = fa.fwd(q, k, v, **kw)
    clean()
    ref_args = (inp.cu_seqlens.tolist(), causal, scale, cap, slopes, begin, end)
    r = osh.forward(inp.q, inp.k, inp.v, *ref_args)
    e = score_error(inp.q, inp.k, scale, cap, slopes, N, dtype)
    h = HALF if dtype == "bf16" else 2.0 ** -23
    lse_ht = f64(lse) if varlen else f64(lse).transpose(1, 0, 2).reshape(H, T)
    inside("LSE", lse_ht, r.lse, e)
    inside("O", f64(o).reshape(T, H, D), r.o,
           (h * (1 + 2 * h) + 2 * e) * (r.o_abs + np.abs(r.o)) + h * np.abs(r.o))
    if backward:
        got = fa.bwd(do, q, k, v, o, lse, **kw)
        clean()
        b = osh.backward(inp.q, inp.k, inp.v, inp.do, *ref_args)
        dq, dk, dv = (f64(x).reshape(y.shape) for x, y in zip(got, (b.dq, b.dk, b.dv)))
        # 2e also covers the sums of dO V^T and dO.O in fp32, D 2^-24 of their terms.
        tiny = (e + D * 2.0 ** -23)
        inside("dV", dv, b.dv, (h + 2 * e) * b.dv_abs + h * np.abs(b.dv))
        c = 2.0 ** -20 if cap else 0.0
        f = 2.0 ** -39 if dtype == "bf16" else 0.0
        inside("dQ", dq, b.dq, f * b.dq_one + c * b.dq_raw + (2 * h + 4 * e) * b.dq_abs + (h + 2 * tiny) * b.dq_del +
               h * np.abs(b.dq))
        inside("dK", dk, b.dk, f * b.dk_one + c * b.dk_raw + (2 * h + 4 * e) * b.dk_abs + (h + 2 * tiny) * b.dk_del +
               h * np.abs(b.dk))
    return o, lse


MASKS = ["none", "docs", "prefix", "window", "any"]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("cap,alibi", [(30.0, False), (0.0, True), (5.0, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_bf16_dense(D, cap, alibi, causal, mask):
    run_case(1 + D, "bf16", [330, 330], 4, 2, D, False, causal, cap, alibi, mask,
             std=2.0 if cap else 1.0)


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("D,H,H_kv", [(64, 6, 3), (128, 8, 1), (128, 5, 5)])
def test_bf16_packed(D, H, H_kv, mask):
    run_case(7 + H, "bf16", [1, 0, 129, 256, 3, 700, 128, 127], H, H_kv, D, True, mask != "prefix",
             20.0, H != 6, mask, std=1.5)


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513])
def test_bf16_lengths(n):
    for D in (64, 128):
        run_case(n, "bf16", [n], 2, 1, D, False, True, 50.0, True, "none")


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("D,H,H_kv,n", [(64, 4, 2, 130), (17, 2, 1, 70), (128, 3, 3, 65),
                                        (1, 1, 1, 33), (40, 4, 1, 1)])
def test_f32(D, H, H_kv, n, mask):
    run_case(D, "f32", [n, n], H, H_kv, D, False, mask == "any", 7.0, True, mask)


@pytest.mark.parametrize("mask,causal", [("docs", True), ("window", False), ("prefix", False), ("none", True)])
def test_f32_more_queries_than_one_look(mask, causal):
    # The backward looks at 1024 queries' ranges at a time, and takes another form when
    # there are many key rows.
    for H, H_kv in ((2, 1), (6, 3)):
        run_case(5 + H, "f32", [1100], H, H_kv, 16, False, causal, 7.0, True, mask)


def test_f32_packed():
    run_case(3, "f32", [5, 0, 90, 1, 33], 4, 2, 32, True, True, 0.0, True, "any")


@pytest.mark.parametrize("std,scale", [(1.0, None), (4.0, None), (9.0, 1.0)])
@pytest.mark.parametrize("D", [64, 128])
def test_cap_far_into_saturation(D, std, scale):
    # Logits from well inside the cap to many times it; the steep part of tanh
    # and its flat part both occur.
    run_case(int(std), "bf16", [200], 2, 2, D, False, True, 10.0, False, "none", std=std,
             scale=scale)


@pytest.mark.parametrize("cap", [1e-3, 1.0, 62.0, 70.0, 300.0, 1e5])
@pytest.mark.parametrize("D", [64, 128])
def test_caps_of_every_size(D, cap):
    # Below and above the size up to which the forward needs no running maximum; logits of
    # std 4 and, at a scale of 2, far over 100.
    run_case(11, "bf16", [300], 2, 1, D, False, True, cap, False, "none", std=2.0)
    run_case(12, "bf16", [300], 2, 1, D, False, False, cap, False, "any", std=2.0, scale=2.0)


@pytest.mark.parametrize("cap", [1e5, 1e8, 1e12, 2.0 ** 100])
@pytest.mark.parametrize("D", [64, 128])
def test_logits_far_below_a_large_cap(D, cap):
    # tanh leaves them as they are to fp32, (x / cap)^2 / 3 < 2^-26: the bounds are those
    # of scores without a cap, but for 2^-22 z of the polynomial.
    n, H, scale = 300, 2, D ** -0.5
    g = torch.Generator().manual_seed(D)
    q, k, v, do = (torch.randn((n, H, D), generator=g).bfloat16() for _ in range(4))
    up = [x.cuda()[None] for x in (q, k, v, do)]
    kw = dict(causal=True, softcap=cap)
    o, lse = fa.fwd(*up[:3], **kw)
    dq = fa.bwd(up[3], *up[:3], o, lse, **kw)[0]
    w = torch.zeros(1, H, n, device="cuda")
    od, ld = fa.decode(q[-1:].cuda(), k.cuda(), v.cuda(), torch.tensor([n], dtype=torch.int32).cuda(),
                       q_len=1, max_seqlen_k=n, softcap=cap, key_weights=w)
    clean()
    r = osh.forward(q, k, v, [0, n], True, scale, cap)
    e = score_error(q, k, scale, 0.0, None, n, "bf16")
    inside("LSE", f64(lse)[0], r.lse, e)
    inside("O", f64(o)[0], r.o, (HALF + 2 * e) * r.o_abs + HALF * np.abs(r.o))
    b = osh.backward(q, k, v, do, [0, n], True, scale, cap)
    inside("dQ", f64(dq)[0], b.dq, (2 * HALF + 4 * e) * b.dq_abs + (HALF + 2 * e) * b.dq_del +
           HALF * np.abs(b.dq) + 2.0 ** -20 * b.dq_raw + 2.0 ** -39 * b.dq_one)
    ro, rl, ra, rw = osh.decode(q[-1:], k, v, [n], q_len=1, scale=scale, page_size=n, cap=cap)
    inside("decode O", f64(od), ro, (HALF + 2 * e) * ra + HALF * np.abs(ro))
    inside("decode LSE", f64(ld), rl, e)
    inside("weights", f64(w), rw, 2 * e * rw + 2.0 ** -22 * (1 + rw))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_rows_all_at_one_end_of_the_cap(D, sign):
    # Every score of a row saturates at the same end: P sits at an end of its range.
    n, H, cap = 260, 2, 60.0
    g = torch.Generator().manual_seed(3)
    q = torch.randn((n, H, D), generator=g).abs() * 8
    k = sign * torch.randn((n, H, D), generator=g).abs() * 8
    v = torch.randn((n, H, D), generator=g)
    q, k, v = (x.bfloat16() for x in (q, k, v))
    o, lse = fa.fwd(*(x.cuda()[None] for x in (q, k, v)), causal=True, softcap=cap, scale=1.0)
    clean()
    r = osh.forward(q, k, v, [0, n], True, 1.0, cap)
    e = score_error(q, k, 1.0, cap, None, n, "bf16")
    inside("LSE", f64(lse)[0], r.lse, e)
    inside("O", f64(o)[0], r.o, (HALF + 2 * e) * r.o_abs + HALF * np.abs(r.o))


@pytest.mark.parametrize("cap,alibi", [(30.0, False), (0.0, True), (5.0, True), (0.0, False)])
@pytest.mark.parametrize("D", [64, 128])
def test_a_row_with_one_key_is_its_value(D, cap, alibi):
    # Whatever P is rounded to, O = P v / P: v to the rounding of the division (2^-23), so
    # the same bf16.
    n, H = 300, 2
    q, k, v = (torch.randn(1, n, H, D, device="cuda").bfloat16() * 2 for _ in range(3))
    slopes = torch.tensor([0.3, 0.1], device="cuda") if alibi else None
    g = torch.Generator().manual_seed(4)
    at = torch.randint(0, n, (1, n), generator=g, dtype=torch.int32).cuda()
    o, _ = fa.fwd(q, k, v, softcap=cap or None, alibi_slopes=slopes, key_begin=at, key_end=at + 1)
    clean()
    assert torch.equal(o[0], v[0, at[0].long()])


def test_ranges_that_see_nothing():
    q = torch.randn(2, 200, 4, 64, device="cuda", dtype=torch.bfloat16)
    z = torch.zeros(2, 200, dtype=torch.int32, device="cuda")
    o, lse = fa.fwd(q, q, q, key_begin=z, key_end=z)
    got = fa.bwd(q, q, q, q, o, lse, key_begin=z, key_end=z)
    clean()
    assert (o == 0).all() and torch.isneginf(lse).all()
    assert all((x == 0).all() for x in got)


def test_ranges_equal_to_the_plain_masks_give_the_plain_result():
    # A full range and causal: the same attention by another path.
    q, k, v = (torch.randn(2, 300, 4, 128, device="cuda", dtype=torch.bfloat16) for _ in range(3))
    z = torch.zeros(2, 300, dtype=torch.int32, device="cuda")
    o, lse = fa.fwd(q, k, v, causal=True, key_begin=z)
    o2, lse2 = fa.fwd(q, k, v, causal=True)
    clean()
    assert (lse - lse2).abs().max() < 1e-4
    assert ((o.float() - o2.float()).abs() <= 2 ** -7 * o2.float().abs() + 2 ** -7).all()


@pytest.mark.parametrize("window", [0, 1, 7, 5000])
@pytest.mark.parametrize("docs,prefix", [(False, False), (True, False), (False, True), (True, True)])
@pytest.mark.parametrize("causal", [True, False])
def test_key_ranges(causal, docs, prefix, window):
    if prefix and not causal:
        return
    lengths = [1, 0, 5, 1030, 2049]
    rng = np.random.default_rng(window)
    ids = (rng.random(sum(lengths)) < 0.02).cumsum().astype(np.int32) if docs else None
    pre = rng.integers(0, 1500, len(lengths)).astype(np.int32) if prefix else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    up = lambda a: None if a is None else torch.from_numpy(a).cuda()
    b, e = fa.key_ranges(sum(lengths), cu_seqlens=cu, max_seqlen=2049, causal=causal,
                         doc_ids=up(ids), prefix_lens=up(pre), window=window or None)
    rb, re = osh.key_ranges(lengths, causal, ids, pre, window)
    clean()
    assert np.array_equal(b.cpu().numpy(), rb) and np.array_equal(e.cpu().numpy(), re)
    if docs:   # dense, the same documents
        d, de = fa.key_ranges(doc_ids=up(ids[6:1036].reshape(2, 515)), causal=causal,
                              window=window or None)
        rb, re = osh.key_ranges([515, 515], causal, ids[6:1036], None, window)
        assert np.array_equal(d.cpu().numpy().ravel(), rb) and np.array_equal(de.cpu().numpy().ravel(), re)


# ------------------------------------------------------------------ decode ---

def run_decode(seed, lengths, q_len, H, H_kv, D, page=None, causal=True, cap=0.0, alibi=False,
               window=0, positions=False, weights=True, std=1.0, max_len=None):
    c = decode_case(seed, dtype="bf16", lengths=lengths, q_len=q_len, H=H, H_kv=H_kv, D=D,
                    page_size=page)
    c.q = c.q * std
    rng = np.random.default_rng(seed)
    B, most = len(lengths), max(max(lengths), 1) if max_len is None else max_len
    slots = most + 3
    slopes = torch.tensor([0.5 * 0.8 ** h for h in range(H)]) if alibi else None
    pos = None
    if positions:
        pos = np.sort(np.stack([[rng.permutation(2 * slots)[:slots] for _ in range(H_kv)]
                                for _ in range(B)]), -1).astype(np.int32)
    w0 = torch.rand(B, H_kv, slots, generator=torch.Generator().manual_seed(seed))
    w = w0.cuda() if weights else None
    up = lambda t: None if t is None else t.cuda()
    if c.block_table is None:
        c.page_size = c.k_cache.shape[0] // B
    o, lse = fa.decode(c.q.cuda(), c.k_cache.cuda(), c.v_cache.cuda(), c.cache_seqlens.cuda(),
                       q_len=q_len, max_seqlen_k=most if page else min(most, c.page_size),
                       block_table=up(c.block_table), page_size=c.page_size, causal=causal,
                       softcap=cap or None, alibi_slopes=up(slopes), window=window or None,
                       key_positions=None if pos is None else torch.from_numpy(pos).cuda(),
                       key_weights=w)
    clean()
    ro, rl, ra, rw = osh.decode(c.q, c.k_cache, c.v_cache, lengths, q_len=q_len, scale=D ** -0.5,
                                causal=causal, page_size=c.page_size, block_table=c.block_table,
                                cap=cap, slopes=slopes, window=window, positions=pos, slots=slots)
    used = torch.isfinite(c.k_cache[:, 0, 0].float())
    e = score_error(c.q, c.k_cache[used], D ** -0.5, cap, slopes, 2 * slots, "bf16")
    inside("LSE", f64(lse), rl, e)
    inside("O", f64(o), ro, (HALF + 2 * e) * ra + HALF * np.abs(ro))
    if weights:
        # each weight is exp of a score and an LSE, both off by e, and no bf16
        inside("weights", f64(w), f64(w0) + rw, 2 * e * rw + 2.0 ** -22 * (1 + rw))


LENS = [1, 127, 128, 129, 0, 1000, 255, 256, 2049, 40, 7]


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("q_len,H,H_kv", [(1, 2, 2), (1, 8, 2), (3, 15, 3), (5, 16, 4), (8, 32, 8),
                                          (9, 21, 3)])
def test_decode_rows(q_len, H, H_kv, D):
    run_decode(q_len * H + D, LENS, q_len, H, H_kv, D, cap=20.0, alibi=H == 8, std=2.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 5, 128, 300])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_window(D, window, causal):
    run_decode(window + D, LENS, 4, 8, 2, D, causal=causal, window=window, alibi=True)
    run_decode(window + D, LENS, 4, 8, 2, D, causal=causal, window=window, cap=8.0, page=64)


@pytest.mark.parametrize("page", [16, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_paged(D, page):
    run_decode(page + D, LENS, 2, 8, 2, D, page=page, cap=20.0, alibi=True)
    run_decode(page + D, LENS, 1, 8, 2, D, page=page, alibi=True, weights=False, window=50)


@pytest.mark.parametrize("window", [0, 40, 400])
def test_decode_positions(window):
    run_decode(window, LENS, 3, 8, 2, 128, positions=True, alibi=True, window=window)
    run_decode(window, LENS, 1, 4, 4, 64, positions=True, cap=10.0, window=window, page=16)


def test_decode_many_sequences_and_few_tiles():
    rng = np.random.default_rng(5)
    run_decode(1, [int(x) for x in rng.integers(0, 900, 70)], 1, 8, 4, 128, cap=30.0, alibi=True)
    run_decode(2, [300, 5, 0, 390], 1, 4, 1, 128, cap=30.0)
    run_decode(3, [300, 5, 0, 390], 1, 4, 1, 64, alibi=True, window=100)
    run_decode(4, [1], 1, 1, 1, 64, cap=30.0)


def test_decode_max_seqlen_above_the_lengths():
    run_decode(9, [100, 300], 1, 8, 2, 128, page=64, cap=30.0, max_len=320)


# ---------------------------------------------------------------- eviction ---

def run_evict(seed, lengths, H_kv, D, keep, recent, page=None, out_page=None, positions=False,
              weights=None, out_slots=None):
    c = decode_case(seed, dtype="bf16", lengths=lengths, q_len=1, H=H_kv, H_kv=H_kv, D=D,
                    page_size=page)
    rng = np.random.default_rng(seed)
    B, most = len(lengths), max(max(lengths), 1)
    slots = most + 2
    w = rng.random((B, H_kv, slots)).astype(np.float32) if weights is None else weights(rng, (B, H_kv, slots))
    pos = rng.integers(0, 1 << 30, (B, H_kv, slots)).astype(np.int32) if positions else None
    if c.block_table is None:
        c.page_size = c.k_cache.shape[0] // B
    kw = {}
    stride = out_table = None
    if out_page:
        n_pages = -(-min(keep, most) // out_page)
        perm = rng.permutation(B * n_pages + 2)[:B * n_pages].reshape(B, n_pages).astype(np.int32)
        out_table, rows = perm, (B * n_pages + 2) * out_page
        kw = dict(out_block_table=torch.from_numpy(perm).cuda(), out_page_size=out_page)
    else:
        stride = keep + 1
        rows = B * stride
    fill = lambda: torch.full((rows, H_kv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ko, vo, n_out, w_out, p_out = fa.evict(
        c.k_cache.cuda(), c.v_cache.cuda(), c.cache_seqlens.cuda(), torch.from_numpy(w).cuda(),
        keep=keep, recent=recent, max_seqlen_k=most if page else c.page_size,
        block_table=None if c.block_table is None else c.block_table.cuda(),
        page_size=c.page_size, key_positions=None if pos is None else torch.from_numpy(pos).cuda(),
        k_out=fill(), v_out=fill(), out_slots=out_slots, **kw)
    clean()
    rk, rv = (torch.full((rows, H_kv, D), 7.0, dtype=torch.bfloat16) for _ in range(2))
    S = out_slots or keep
    rw, rp = np.zeros((B, H_kv, S), np.float32), np.full((B, H_kv, S), -1, np.int32)
    for b, n in enumerate(lengths):
        at = osh.cache_rows(b, n, c.page_size, c.block_table)
        for h in range(H_kv):
            s = osh.kept_slots(w[b, h], n, keep, recent)
            to = osh.cache_rows(b, len(s), out_page or stride, out_table)
            rk[to, h], rv[to, h] = c.k_cache[at[s], h], c.v_cache[at[s], h]
            rw[b, h, :len(s)] = w[b, h, s]
            rp[b, h, :len(s)] = s if pos is None else pos[b, h, s]
    assert n_out.cpu().tolist() == [min(n, keep) for n in lengths]
    assert np.array_equal(p_out.cpu().numpy(), rp)
    assert np.array_equal(w_out.cpu().numpy(), rw, equal_nan=True)
    assert torch.equal(ko.cpu(), rk) and torch.equal(vo.cpu(), rv)


@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (100, 0), (100, 17), (128, 128), (3000, 5)])
@pytest.mark.parametrize("D,page,out_page", [(128, None, None), (64, 16, None), (128, 64, 128),
                                             (64, 256, 16), (8, None, 64)])
def test_evict(D, page, out_page, keep, recent):
    run_evict(keep + D, LENS + [2500], 3, D, keep, recent, page, out_page)


@pytest.mark.parametrize("kind", ["equal", "few", "odd", "tiny"])
def test_evict_weights_with_ties_and_oddities(kind):
    def weights(rng, shape):
        if kind == "equal":
            return np.full(shape, 0.25, np.float32)
        if kind == "few":
            return rng.integers(0, 3, shape).astype(np.float32)
        if kind == "tiny":
            return rng.random(shape).astype(np.float32) * 1e-42
        w = rng.standard_normal(shape).astype(np.float32)
        w[rng.random(shape) < 0.2] = np.nan
        w[rng.random(shape) < 0.1] = np.inf
        w[rng.random(shape) < 0.1] = -np.inf
        w[rng.random(shape) < 0.1] = -0.0
        w[rng.random(shape) < 0.1] = 0.0
        return w
    for keep, recent in ((200, 0), (200, 33), (1500, 3)):
        run_evict(4, [2000, 199, 1501, 0, 300], 2, 64, keep, recent, weights=weights)


@pytest.mark.parametrize("kind", ["random", "few"])
def test_evict_more_slots_than_shared_memory_holds(kind):
    w = (lambda rng, s: rng.integers(0, 5, s).astype(np.float32)) if kind == "few" else None
    run_evict(21, [60001, 49152, 50000, 7], 1, 16, 9000, 100, weights=w)


@pytest.mark.parametrize("keep", [1, 2047, 2048, 2049, 4000, 8191])
def test_evict_at_the_size_of_the_gathered_list(keep):
    # Two values only, or all of one binade: more keys share a digit than the list holds.
    run_evict(22, [8192, 8191], 2, 8, keep, 0,
              weights=lambda rng, s: 1 + rng.integers(0, 2, s).astype(np.float32) * 2.0 ** -23)
    run_evict(23, [8192, 5000], 1, 8, keep, 1,
              weights=lambda rng, s: (1 + rng.random(s) / 1024).astype(np.float32))


def test_evict_positions_and_room_for_new_tokens():
    run_evict(8, [700, 30], 2, 128, 100, 10, positions=True, out_slots=160)


def test_evict_into_the_same_pool():
    # 4 pages read, 2 other pages written.
    pool_k, pool_v = (torch.randn(10 * 64, 2, 64, device="cuda").bfloat16() for _ in range(2))
    table = torch.tensor([[7, 2, 9, 4]], dtype=torch.int32, device="cuda")
    out = torch.tensor([[0, 5]], dtype=torch.int32, device="cuda")
    w = torch.rand(1, 2, 256, device="cuda")
    old = pool_k.clone()
    k2, _, n, _, pos = fa.evict(pool_k, pool_v, torch.tensor([250], dtype=torch.int32, device="cuda"),
                                w, keep=100, recent=8, max_seqlen_k=250, block_table=table,
                                page_size=64, k_out=pool_k, v_out=pool_v, out_block_table=out,
                                out_page_size=64)
    clean()
    assert k2.data_ptr() == pool_k.data_ptr() and n.item() == 100
    for h in range(2):
        s = pos[0, h].long()
        src = old[table[0].long()[s // 64] * 64 + s % 64, h]
        i = torch.arange(100, device="cuda")
        assert torch.equal(pool_k[out[0].long()[i // 64] * 64 + i % 64, h], src)
    untouched = [7, 2, 9, 4, 1, 3, 6, 8]
    assert all(torch.equal(pool_k[p * 64:p * 64 + 64], old[p * 64:p * 64 + 64]) for p in untouched)


def test_bad_lengths_and_pages_are_reported_not_read():
    k, v = (torch.randn(2 * 64, 2, 64, device="cuda").bfloat16() for _ in range(2))
    q = torch.randn(2, 4, 64, device="cuda").bfloat16()
    w = torch.zeros(2, 2, 128, device="cuda")
    table = torch.tensor([[0, 1], [1, 50]], dtype=torch.int32, device="cuda")
    for lens in ([128, 129], [-1, 5], [10, 100]):   # too long, negative, page 50 of 2
        n = torch.tensor(lens, dtype=torch.int32, device="cuda")
        fa.decode(q, k, v, n, q_len=1, max_seqlen_k=128, block_table=table, page_size=64,
                  softcap=30.0, key_weights=w)
        assert fa.check_device_error()[0] != 0
        fa.evict(k, v, n, w, keep=128, recent=0, max_seqlen_k=128, block_table=table, page_size=64)
        assert fa.check_device_error()[0] != 0
    clean()


# ------------------------------------------------- together, streams, graphs ---

def test_prefill_decode_evict_decode():
    # A cache that is filled, read with its weights added up, thinned out and read on.
    n, H, H_kv, D, cap, scale, window = 700, 8, 2, 128, 25.0, 128 ** -0.5, 500
    g = torch.Generator().manual_seed(12)
    new = 3
    q, k, v = (torch.randn((n + new, h, D), generator=g).bfloat16() * 2 for h in (H, H_kv, H_kv))
    slopes = torch.tensor([0.02 * 0.8 ** h for h in range(H)])
    begin = np.maximum(0, np.arange(n) - window + 1).astype(np.int32)
    up = lambda t: t.cuda()
    shape = dict(softcap=cap, alibi_slopes=up(slopes))
    # prefill
    o, lse = fa.fwd(up(q[:n])[None], up(k[:n])[None], up(v[:n])[None], causal=True,
                    key_begin=up(torch.from_numpy(begin))[None], **shape)
    r = osh.forward(q[:n], k[:n], v[:n], [0, n], True, scale, cap, slopes, begin)
    e = score_error(q, k, scale, cap, slopes, n + new, "bf16")
    inside("prefill O", f64(o)[0], r.o, (HALF + 2 * e) * r.o_abs + HALF * np.abs(r.o))
    # the last 8 tokens again as a decode step: the weights they give to the cache
    room = 256
    lens = torch.tensor([n], dtype=torch.int32).cuda()
    w = torch.zeros(1, H_kv, n, device="cuda")
    o8, _ = fa.decode(up(q[n - 8:n]), up(k[:n]), up(v[:n]), lens, q_len=8, max_seqlen_k=n,
                      window=window, key_weights=w, **shape)
    inside("decode O", f64(o8), r.o[-8:], (HALF + 2 * e) * r.o_abs[-8:] + HALF * np.abs(r.o[-8:]))
    # keep 200 of 700, room for new tokens
    k2, v2, n2, w2, pos = fa.evict(up(k[:n]), up(v[:n]), lens, w, keep=200, recent=32,
                                   max_seqlen_k=n, out_slots=room)
    assert n2.tolist() == [200]
    # three more tokens, one at a time, in slots 200 .. with positions 700 ..
    held = [osh.kept_slots(w[0, h].cpu().numpy(), n, 200, 32) for h in range(H_kv)]
    w_ref = np.zeros((H_kv, room))
    for h in range(H_kv):
        w_ref[h, :200] = w[0, h].cpu().numpy()[held[h]]
    for t in range(new):
        s = 200 + t
        k2[s], v2[s] = up(k[n + t]), up(v[n + t])
        pos[:, :, s] = n + t
        o1, _ = fa.decode(up(q[n + t:n + t + 1]), k2, v2, n2 + t + 1, q_len=1, max_seqlen_k=room,
                          window=window, key_positions=pos, key_weights=w2, **shape)
        for h in range(H_kv):
            at = np.concatenate([held[h], n + np.arange(t + 1)])
            heads = slice(h * H // H_kv, (h + 1) * H // H_kv)
            ro, _, ra, rw = osh.decode(q[n + t:n + t + 1, heads], k[at][:, h:h + 1], v[at][:, h:h + 1],
                                       [s + 1], q_len=1, scale=scale, page_size=s + 1, cap=cap,
                                       slopes=slopes[heads], window=window, positions=at[None, None])
            inside("O after eviction", f64(o1)[:, heads], ro, (HALF + 2 * e) * ra + HALF * np.abs(ro))
            w_ref[h, :s + 1] += rw[0, 0]
    clean()
    inside("weights after eviction", f64(w2)[0], w_ref, 2 * e * w_ref + 2.0 ** -20 * (1 + w_ref))


def _small_state(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    st = dict(q=rnd(1, 300, 4, 64), k=rnd(1, 300, 2, 64), v=rnd(1, 300, 2, 64), do=rnd(1, 300, 4, 64),
              kc=rnd(2 * 400, 2, 64), vc=rnd(2 * 400, 2, 64), qd=rnd(2, 4, 64),
              sl=torch.tensor([0.3, 0.2, 0.1, 0.05], device="cuda"),
              b=torch.zeros(1, 300, dtype=torch.int32, device="cuda"),
              lens=torch.tensor([400, 200], dtype=torch.int32, device="cuda"),
              w=torch.rand(2, 2, 400, generator=g, device="cuda"))
    st["b"][:, 150:] = 100
    return st


def _all_of_it(s):
    kw = dict(causal=True, softcap=20.0, alibi_slopes=s["sl"], key_begin=s["b"])
    o, lse = fa.fwd(s["q"], s["k"], s["v"], **kw)
    grads = fa.bwd(s["do"], s["q"], s["k"], s["v"], o, lse, **kw)
    w = s["w"].clone()
    od, ld = fa.decode(s["qd"], s["kc"], s["vc"], s["lens"], q_len=1, max_seqlen_k=400, softcap=20.0,
                       window=300, key_weights=w)
    return (o, lse, *grads, od, ld, w) + fa.evict(s["kc"], s["vc"], s["lens"], w, keep=100, recent=7,
                                                  max_seqlen_k=400)


def _agree(a, b, exact=True):
    for i, (x, y) in enumerate(zip(a, b)):
        if exact and i != 2:   # dQ: reproducible to rounding
            assert torch.equal(x, y), i
        else:
            assert torch.allclose(x.float(), y.float(), rtol=2 ** -6, atol=2 ** -9), i


def test_same_inputs_same_bits():
    s = _small_state(1)
    _agree(_all_of_it(s), _all_of_it(s))
    clean()


def test_on_another_stream():
    ref = _all_of_it(_small_state(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        busy = torch.randn(3000, 3000, device="cuda") @ torch.randn(3000, 3000, device="cuda")
        got = _all_of_it(_small_state(2))
    side.synchronize()
    assert busy.isfinite().all()
    _agree(got, ref)
    clean()


def test_two_streams_at_once():
    states = [_small_state(3), _small_state(4)]
    refs = [_all_of_it(s) for s in states]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in states]
    got = [None, None]
    for _ in range(5):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = _all_of_it(states[i])
    torch.cuda.synchronize()
    for g, r in zip(got, refs):
        _agree(g, r)
    clean()


def test_captured_and_replayed_with_new_inputs():
    s = _small_state(5)
    _all_of_it(s)   # the first call of each kernel on a device is made outside a capture
    graphs, outs = [], []
    for _ in range(2):   # two graphs of one memory pool
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            outs.append(_all_of_it(s))
        graphs.append(g)
    for seed in (6, 7):
        new = _small_state(seed)
        for n in s:
            s[n].copy_(new[n])
        ref = [x.clone() for x in _all_of_it(new)]
        for g, o in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            _agree(o, ref)
    clean()


def test_debug_build_runs_the_shaped_kernels():
    from exact_io_aware_tmem_b200 import attention, build
    build.build(debug=True)
    s = _small_state(8)
    ref = _all_of_it(s)
    with attention.debug_build():
        got = _all_of_it(s)
        clean()
    _agree(got, ref)


# ------------------------------------------------------------- far and empty ---

def test_pages_before_the_window_may_be_gone():
    # Their block-table entries are invalid and the rows they had hold NaN.
    lengths, window, page = [1000, 300, 90], 130, 64
    c = decode_case(77, dtype="bf16", lengths=lengths, q_len=2, H=4, H_kv=2, D=128, page_size=page)
    ro, rl, ra, rw = osh.decode(c.q, c.k_cache, c.v_cache, lengths, q_len=2, scale=128 ** -0.5,
                                page_size=page, block_table=c.block_table, window=window)
    for b, n in enumerate(lengths):
        for i in range(max(0, n - window - 1) // page):
            blk = int(c.block_table[b, i])
            c.k_cache[blk * page:(blk + 1) * page] = float("nan")
            c.v_cache[blk * page:(blk + 1) * page] = float("nan")
            c.block_table[b, i] = -1
    w = torch.zeros(3, 2, 1000, device="cuda")
    o, lse = fa.decode(c.q.cuda(), c.k_cache.cuda(), c.v_cache.cuda(), c.cache_seqlens.cuda(), q_len=2,
                       max_seqlen_k=1000, block_table=c.block_table.cuda(), page_size=page,
                       window=window, key_weights=w)
    clean()
    inside("O", f64(o), ro, (HALF + 4e-4) * ra + HALF * np.abs(ro))
    inside("LSE", f64(lse), rl, 2e-4)
    inside("weights", f64(w), rw, 4e-4 * rw)


def test_cache_rows_past_2_31_elements():
    # 2.2 million rows of 8 heads of 128: element offsets pass 2^31, byte offsets 2^32.
    rows, H_kv, D, page, n = 2_200_064, 8, 128, 64, 500
    k, v = (torch.empty(rows, H_kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pages = torch.tensor([[34375, 3, 34370, 34000, 20000, 17, 34373, 33333]], dtype=torch.int32)
    at = osh.cache_rows(0, n, page, pages)
    assert at.max() < rows
    g = torch.Generator().manual_seed(1)
    kk, vv = (torch.randn((n, H_kv, D), generator=g).bfloat16() for _ in range(2))
    idx = torch.from_numpy(at).cuda()
    k[idx], v[idx] = kk.cuda(), vv.cuda()
    q = torch.randn((1, 8, D), generator=g).bfloat16()
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    w = torch.zeros(1, H_kv, n, device="cuda")
    o, lse = fa.decode(q.cuda(), k, v, lens, q_len=1, max_seqlen_k=n, block_table=pages.cuda(),
                       page_size=page, softcap=30.0, key_weights=w)
    ro, rl, ra, rw = osh.decode(q, kk, vv, [n], q_len=1, scale=D ** -0.5, page_size=n, cap=30.0)
    inside("O", f64(o), ro, (HALF + 4e-4) * ra + HALF * np.abs(ro))
    inside("weights", f64(w), rw, 4e-4 * rw)
    out = torch.tensor([[34374, 2]], dtype=torch.int32, device="cuda")
    _, _, n2, _, pos = fa.evict(k, v, lens, w, keep=100, recent=4, max_seqlen_k=n,
                                block_table=pages.cuda(), page_size=page, k_out=k, v_out=v,
                                out_block_table=out, out_page_size=page)
    clean()
    i = torch.arange(100)
    to = out[0].cpu().long()[i // page] * page + i % page
    for h in range(H_kv):
        s = pos[0, h].long().cpu()
        assert torch.equal(k[to.cuda(), h].cpu(), kk[s, h]) and torch.equal(v[to.cuda(), h].cpu(), vv[s, h])


def test_tensors_past_2_31_elements():
    # 270 thousand tokens of 64 heads of 128; each sees its last 40 keys.
    N, H, D, window = 270_000, 64, 128, 40
    g = torch.Generator("cuda").manual_seed(2)
    q = torch.randn((1, N, H, D), generator=g, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn((1, N, 1, D), generator=g, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    begin = (torch.arange(N, device="cuda") - window + 1).clamp(min=0).int()[None]
    kw = dict(causal=True, softcap=30.0, key_begin=begin)
    o, lse = fa.fwd(q, k, v, **kw)
    dq, dk, dv = fa.bwd(q, q, k, v, o, lse, **kw)
    clean()
    m = 300   # the last tokens, from those whose keys lie among them on
    tail = lambda t: t[0, N - m:].cpu()
    qq, kk, vv = tail(q)[:, H - 2:], tail(k), tail(v)
    b = np.maximum(0, np.arange(m) - window + 1)
    r = osh.forward(qq, kk, vv, [0, m], True, D ** -0.5, 30.0, None, b)
    e = score_error(qq, kk, D ** -0.5, 30.0, None, m, "bf16")
    s = slice(window, m)
    inside("O", f64(tail(o)[:, H - 2:])[s], r.o[s], ((HALF + 2 * e) * r.o_abs + HALF * np.abs(r.o))[s])
    d = osh.backward(qq, kk, vv, qq, [0, m], True, D ** -0.5, 30.0, None, b)
    tol = (2 * HALF + 4 * e) * d.dq_abs + (HALF + 2 * e) * d.dq_del + HALF * np.abs(d.dq) + \
        2.0 ** -20 * d.dq_raw + 2.0 ** -39 * d.dq_one
    inside("dQ", f64(tail(dq)[:, H - 2:])[s], d.dq[s], tol[s])
    assert torch.isfinite(dk).all() and torch.isfinite(dv).all()


def test_nothing_to_do():
    e = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt, device="cuda")
    o, lse = fa.fwd(e(2, 0, 4, 64), e(2, 0, 2, 64), e(2, 0, 2, 64), softcap=30.0)
    assert o.shape == (2, 0, 4, 64) and lse.shape == (2, 4, 0)
    i32 = torch.int32
    w = torch.rand(2, 2, 5, device="cuda")
    w0 = w.clone()
    od, ld = fa.decode(e(2, 4, 64) + 1, e(10, 2, 64), e(10, 2, 64), e(2, dt=i32), q_len=1,
                       max_seqlen_k=0, page_size=5, softcap=30.0, key_weights=w)
    assert (od == 0).all() and torch.isneginf(ld).all() and torch.equal(w, w0)
    k2, _, n, w2, pos = fa.evict(e(10, 2, 64), e(10, 2, 64), e(2, dt=i32), w, keep=3, max_seqlen_k=0,
                                 page_size=5)
    assert (n == 0).all() and (w2 == 0).all() and (pos == -1).all() and (k2 == 0).all()
    b, en = fa.key_ranges(0, B=3)
    assert b.shape == (3, 0)
    clean()
