"""Edges of the shaped entry points on the GPU: workspaces in a bad state, values far from
the usual, rows that belong to nobody, recipes of the documentation."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

import exact_io_aware_tmem_b200 as fa
from exact_io_aware_tmem_b200 import _abi
from exact_io_aware_tmem_b200.workloads import decode_case, random_case
from oracle import shaped as osh
from tests._util import f64
from tests.test_shaped_gpu import (HALF, _agree, _all_of_it, _small_state, clean, inside,
                                   score_error)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_io_aware_tmem_b200 import build
    build.build()


# ------------------------------- what a timed-out first kernel leaves behind ---

class _Decode:
    """One decode's arguments; its workspace, and where the segments' first and last
    group lie in it."""

    def __init__(self, D=128, H=8, H_kv=2, lengths=(700, 40)):
        g = torch.Generator("cuda").manual_seed(D)
        rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
        self.B, self.H, self.H_kv, self.D, self.most = len(lengths), H, H_kv, D, max(lengths)
        self.q = rnd(self.B, H, D)
        self.k, self.v = (rnd(self.B * self.most, H_kv, D) for _ in range(2))
        self.lens = torch.tensor(lengths, dtype=torch.int32, device="cuda")
        self.lib = _abi.lib()
        self.need = self.lib.fa_decode_shaped_workspace_size(self.B, 1, H, H_kv, D, self.most, 1)
        self.ws = torch.empty(self.need, dtype=torch.uint8, device="cuda")
        self.w = torch.rand(self.B, H_kv, self.most, generator=g, device="cuda")
        self.groups = torch.cuda.get_device_properties(0).multi_processor_count // H_kv
        up = lambda n: -(-n // 256) * 256
        rows, segs = (self.B + self.groups) * H_kv * (H // H_kv), self.B * H_kv
        at = up(rows * D * 4) + up(rows * 4)
        ints = lambda o: self.ws[o:o + 4 * segs].view(torch.int32)
        self.first, self.last = ints(at), ints(at + up(segs * 4))

    def run(self):
        return fa.decode(self.q, self.k, self.v, self.lens, q_len=1, max_seqlen_k=self.most,
                         softcap=30.0, key_weights=self.w, workspace=self.ws)

    def finish(self, o, lse):
        _abi.check(self.lib.fa_selftest_decode_finish(
            o.data_ptr(), lse.data_ptr(), self.lens.data_ptr(), self.B, 1, self.H, self.H_kv, self.D,
            self.most, self.w.data_ptr(), self.most, self.ws.data_ptr(), self.need,
            torch.cuda.current_stream().cuda_stream), "fa_selftest_decode_finish")


@pytest.mark.parametrize("D", [64, 128])
def test_decode_finish_on_a_sound_workspace_adds_the_weights_again(D):
    d = _Decode(D)
    d.w.zero_()
    o, lse = d.run()
    clean()
    once, o1, lse1 = d.w.clone(), o.clone(), lse.clone()
    assert (d.first >= 0).all() and (d.first <= d.last).all() and (d.last < d.groups).all()
    d.finish(o, lse)
    clean()
    assert torch.equal(d.w, once + once)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)


MOST = 2 ** 31 - 1


@pytest.mark.parametrize("first,last", [(-1, -1), (0, "groups"), (3, 1), (-5, 2), (MOST, MOST),
                                        (-MOST - 1, MOST), ("groups", "groups")])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_finish_reports_pieces_outside_the_workspace(D, first, last):
    d = _Decode(D)
    d.ws.fill_(0xFF)   # NaN, -1
    d.first.fill_(d.groups if first == "groups" else first)
    d.last.fill_(d.groups if last == "groups" else last)
    o = torch.full((d.B, d.H, D), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((d.B, d.H), 5.0, device="cuda")
    w0 = d.w.clone()
    d.finish(o, lse)
    st, where = fa.check_device_error()
    assert st == _abi.FA_ERR_INVALID_ARG and where == 0xE0F03
    assert torch.equal(d.w, w0) and (o == 3.0).all() and (lse == 5.0).all()
    clean()


# ------------------------------------------------------- values far from one ---

@pytest.mark.parametrize("log2_v", [50, -20])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("cap,alibi", [(1.0, False), (10.0, False), (44.0, False), (45.0, False),
                                       (51.0, False), (52.0, False), (62.0, False), (200.0, False),
                                       (20.0, True), (0.0, True)])
@pytest.mark.parametrize("D", [64, 128])
def test_large_and_small_values_at_either_end_of_the_cap(D, cap, alibi, sign, log2_v):
    # Every score of a row at the same end of the cap. 300 keys of |v| below 2^53: less than
    # 2^62 in all. The bounds are relative to |v|, as everywhere.
    n, H = 300, 2
    g = torch.Generator().manual_seed(5)
    q = torch.randn((n, H, D), generator=g).abs() * 8
    k = sign * torch.randn((n, H, D), generator=g).abs() * 8
    v = torch.randn((n, H, D), generator=g) * 2.0 ** log2_v
    q, k, v = (x.bfloat16() for x in (q, k, v))
    scale = 1.0 if cap else 2.0 ** -10
    slopes = torch.tensor([0.3, 0.1]) if alibi else None
    o, lse = fa.fwd(*(x.cuda()[None] for x in (q, k, v)), causal=True, softcap=cap or None, scale=scale,
                    alibi_slopes=None if slopes is None else slopes.cuda())
    clean()
    r = osh.forward(q, k, v, [0, n], True, scale, cap, slopes)
    e = score_error(q, k, scale, cap, slopes, n, "bf16")
    if cap:
        # The part of e that is the product's error, D 2^-24 scale |q||k|, reaches z by 1 - tanh^2
        # <= 4 e^(-2 u).
        dot = D * 2.0 ** -24 * scale * (abs(f64(q)).max(0) ** 2).sum(-1).max() ** 0.5 * \
            (abs(f64(k)).max(0) ** 2).sum(-1).max() ** 0.5
        low = min(abs(scale * f64(q)[:, h] @ f64(k)[:, h].T).min() for h in range(H))
        z = cap + (0.0 if slopes is None else float(slopes.max()) * n)
        e = dot * 4 * np.exp(-2 * low / cap) + 2.0 ** -21 * (2 + z + cap) + 1e-4
    inside("LSE", f64(lse)[0], r.lse, e)
    # As in the masked tiles of other cases: the P that are summed are the rounded ones.
    inside("O", f64(o)[0], r.o, (HALF * (1 + 2 * HALF) + 2 * e) * (r.o_abs + abs(r.o)) + HALF * abs(r.o))


# ------------------------------------------------------ rows that are nobody's ---

@pytest.mark.parametrize("page", [None, 64])
@pytest.mark.parametrize("q_len,window,alibi", [(1, 0, False), (5, 0, True), (2, 100, False)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_bits_do_not_depend_on_rows_past_the_end(D, q_len, window, alibi, page):
    # Stale tokens, or anything else, behind a sequence's length: the results are the same bits.
    g = torch.Generator("cuda").manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    lengths, most = [70, 300, 129], 448
    q, k, v = rnd(3 * q_len, 8, D), rnd(3 * most, 2, D), rnd(3 * most, 2, D)
    kw = dict(q_len=q_len, max_seqlen_k=most, softcap=30.0, window=window or None,
              page_size=page or most)
    if page:
        kw["block_table"] = torch.arange(3 * most // page, dtype=torch.int32, device="cuda").view(3, -1)
    if alibi:
        kw["alibi_slopes"] = torch.linspace(0.01, 0.2, 8, device="cuda")
    outs = []
    for fill in (0.0, 1.0, 100.0, float("inf"), float("nan")):
        for b, n in enumerate(lengths):
            k[b * most + n:(b + 1) * most] = fill
            v[b * most + n:(b + 1) * most] = fill
        w = torch.zeros(3, 2, most, device="cuda")
        outs.append((*fa.decode(q, k, v, torch.tensor(lengths, dtype=torch.int32, device="cuda"),
                                key_weights=w, **kw), w))
        clean()
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))


@pytest.mark.parametrize("page_id", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 25, 4, -1, -2 ** 31])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(), dict(n_split=2)])
def test_pages_outside_the_cache_are_reported(kw, page_id):
    # Every id outside [0, 4), those whose first row leaves 32 bits among them; the shaped,
    # the balanced and the split decode.
    q = torch.randn(1, 4, 128, device="cuda").bfloat16()
    k, v = (torch.randn(4 * 64, 2, 128, device="cuda").bfloat16() for _ in range(2))
    lens = torch.tensor([200], dtype=torch.int32, device="cuda")
    for bad in range(4):
        table = torch.arange(4, dtype=torch.int32, device="cuda")[None]
        table[0, bad] = page_id
        fa.decode(q, k, v, lens, q_len=1, max_seqlen_k=256, block_table=table, page_size=64, **kw)
        assert fa.check_device_error()[0] == _abi.FA_ERR_INVALID_ARG
    clean()


@pytest.mark.parametrize("D", [64, 128])
def test_decode_bits_do_not_depend_on_pages_before_the_window(D):
    # The pages that no query sees hold large keys, or have been given back.
    n, window, page = 700, 100, 16
    g = torch.Generator("cuda").manual_seed(D)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, k, v = rnd(2, 8, D), rnd(704, 2, D), rnd(704, 2, D)
    gone = (n - window - 1) // page   # pages of slots that neither of the two queries sees
    k[:gone * page] = 100.0
    table = torch.arange(704 // page, dtype=torch.int32, device="cuda")[None]
    freed = table.clone()
    freed[:, :gone] = -1
    outs = []
    for t in (table, freed):
        w = torch.zeros(1, 2, n, device="cuda")
        outs.append((*fa.decode(q, k, v, torch.tensor([n], dtype=torch.int32, device="cuda"), q_len=2,
                                max_seqlen_k=n, block_table=t, page_size=page, window=window,
                                softcap=30.0, key_weights=w), w))
        clean()
    assert all(torch.equal(x, y) for x, y in zip(*outs))


# ------------------------------------------------------ workspace under a window ---

@pytest.mark.parametrize("window,q_len", [(1, 1), (100, 1), (129, 8), (3000, 2), (1 << 30, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_window_needs_room_for_its_slots_only(D, window, q_len):
    # The size that the header gives for a window, and not a byte behind it.
    B, H, H_kv, most = 3, 8, 2, 4000
    g = torch.Generator("cuda").manual_seed(window % 97)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    q, k, v = rnd(B * q_len, H, D), rnd(B * most, H_kv, D), rnd(B * most, H_kv, D)
    lens = torch.tensor([most, 130, 2049], dtype=torch.int32, device="cuda")
    lib, span = _abi.lib(), min(most, window + q_len + 127)
    need = lib.fa_decode_shaped_workspace_size(B, q_len, H, H_kv, D, span, 1)
    ws = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    w, w2 = (torch.zeros(B, H_kv, most, device="cuda") for _ in range(2))
    o, lse = torch.empty_like(q), torch.empty(B * q_len, H, device="cuda")
    shape = _abi.DecodeShape(30.0, None, window, None, w.data_ptr(), most)
    args = (q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), lens.data_ptr(), None,
            B, q_len, H, H_kv, D, most, 0, B * most, most, 1, -1.0, ctypes.byref(shape), ws.data_ptr())
    stream = torch.cuda.current_stream().cuda_stream
    assert lib.fa_decode_shaped(*args, need - 1, stream) == _abi.FA_ERR_INVALID_ARG
    assert lib.fa_decode_shaped(*args, need, stream) == _abi.FA_OK
    clean()
    assert (ws[need:] == 0xA5).all()
    big = torch.empty(lib.fa_decode_shaped_workspace_size(B, q_len, H, H_kv, D, most, 1),
                      dtype=torch.uint8, device="cuda")
    o2, lse2 = fa.decode(q, k, v, lens, q_len=q_len, max_seqlen_k=most, softcap=30.0, window=window,
                         key_weights=w2, workspace=big)
    clean()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(w, w2)
    # every query's weights add up to one
    assert torch.allclose(w.sum(-1), torch.tensor(float(q_len * H // H_kv), device="cuda"), rtol=1e-3)


def test_decode_window_allocates_for_its_slots_only():
    B, H, H_kv, D, most, window = 4, 16, 2, 64, 32768, 200
    q = torch.randn(B * 8, H, D, device="cuda").bfloat16()
    k, v = (torch.zeros(B * most, H_kv, D, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    lens = torch.full((B,), most, dtype=torch.int32, device="cuda")
    w = torch.zeros(B, H_kv, most, device="cuda")
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    out = fa.decode(q, k, v, lens, q_len=8, max_seqlen_k=most, softcap=30.0, window=window, key_weights=w)
    clean()
    used = torch.cuda.max_memory_allocated() - before
    size = lambda n: _abi.lib().fa_decode_shaped_workspace_size(B, 8, H, H_kv, D, n, 1)
    results = sum(x.numel() * x.element_size() for x in out)
    assert used <= size(window + 8 + 127) + results + 4096 < size(most) // 4


# -------------------------------------------------------------- the README ---

def test_readme_of_shaped_scores_on_sequences_of_different_lengths():
    # Its code as it stands, over two sequences of which one is shorter than what is kept.
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "README.md")).read()
    code, = [c for c in re.findall(r"```python\n(.*?)```", text, re.S) if "fa.evict(" in c]
    B, H, H_kv, D, N, keep, recent, cap = 2, 4, 2, 64, 200, 2048, 64, 50.0
    lengths, max_len = [2500, 700], 2600
    g = torch.Generator().manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=g).bfloat16() * 2
    t = dict(q=rnd(B, N, H, D), k=rnd(B, N, H_kv, D), v=rnd(B, N, H_kv, D), dout=rnd(B, N, H, D),
             slopes=torch.full((H,), 0.1), ids=torch.arange(B * N, dtype=torch.int32).view(B, N) // 70,
             k_cache=rnd(B * max_len, H_kv, D), v_cache=rnd(B * max_len, H_kv, D), q_last=rnd(B, H, D),
             lens=torch.tensor(lengths, dtype=torch.int32), q_new=rnd(B, H, D), k_new=rnd(B, H_kv, D),
             v_new=rnd(B, H_kv, D))
    names = {n: x.cuda() for n, x in t.items()}
    names.update(torch=torch, B=B, H_kv=H_kv, max_len=max_len)
    exec(code, names)
    clean()
    e = score_error(torch.cat([t["q_new"], t["q_last"]]), torch.cat([t["k_cache"], t["k_new"]]), D ** -0.5,
                    cap, None, max_len, "bf16")
    assert names["lens2"].tolist() == [keep + 1, 701]
    pos, w = names["pos2"].cpu(), names["w"].cpu().numpy()
    for b, n in enumerate(lengths):
        m = int(names["lens2"][b])
        for h in range(H_kv):
            at = osh.kept_slots(w[b, h], n, keep, recent)
            assert pos[b, h, :m].tolist() == at.tolist() + [n] and (pos[b, h, m:] == -1).all()
            kk = torch.cat([t["k_cache"][b * max_len + at][:, h:h + 1], t["k_new"][b, h:h + 1][None]])
            vv = torch.cat([t["v_cache"][b * max_len + at][:, h:h + 1], t["v_new"][b, h:h + 1][None]])
            heads = slice(h * H // H_kv, (h + 1) * H // H_kv)
            ro, rl, ra, rw = osh.decode(t["q_new"][b:b + 1, heads], kk, vv, [m], q_len=1, scale=D ** -0.5,
                                        page_size=m, cap=cap, positions=pos[b:b + 1, h:h + 1, :m].numpy())
            inside("O", f64(names["o"])[b:b + 1, heads], ro, (HALF + 2 * e) * ra + HALF * abs(ro))
            inside("LSE", f64(names["lse"])[b:b + 1, heads], rl, e)
            w0 = np.concatenate([w[b, h][at].astype(np.float64), [0.0]])
            inside("weights", f64(names["w2"])[b, h, :m], w0 + rw[0, 0],
                   2 * e * rw[0, 0] + 2.0 ** -22 * (1 + w0 + rw[0, 0]))


# ------------------------------------------------------------------ streams ---

def test_stream_by_either_name(monkeypatch):
    from exact_io_aware_tmem_b200 import attention
    dev, side = torch.device("cuda", 0), torch.cuda.Stream()
    for stream in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(stream):
            ours = attention._stream(dev)
            with monkeypatch.context() as m:
                m.setattr(attention, "_raw_stream", None)
                assert attention._stream(dev) == ours == stream.cuda_stream


def test_a_small_wait_budget_is_raised():
    # No wait of these calls lasts ten milliseconds: all of them succeed.
    s = _small_state(11)
    _all_of_it(s)
    clean()
    fa.set_wait_budget(1)
    try:
        got = _all_of_it(s)
        clean()
    finally:
        fa.set_wait_budget(0)
    _agree(got, _all_of_it(s))


# ------------------------------------------------------------- negative slopes ---

@pytest.mark.parametrize("steep", [-0.01, -0.2, -2.0])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("dtype,D", [("bf16", 64), ("bf16", 128), ("f32", 40)])
def test_negative_slopes(dtype, D, causal, cap, steep):
    # They favour the far keys: the softmax's reference moves at every tile. One head's slope
    # is positive beside them.
    lengths, H, H_kv = [333, 333], 4, 2
    N, T = 333, 666
    inp = random_case(17, dtype=dtype, lengths=lengths, H=H, H_kv=H_kv, D=D, varlen=False)
    slopes = torch.tensor([steep, 0.5 * steep, -0.3 * steep, 0.1 * steep])
    dev = lambda t: t.cuda().view(2, N, *t.shape[1:]).contiguous()
    kw = dict(causal=causal, softcap=cap or None, alibi_slopes=slopes.cuda())
    q, k, v, do = dev(inp.q), dev(inp.k), dev(inp.v), dev(inp.do)
    o, lse = fa.fwd(q, k, v, **kw)
    got = fa.bwd(do, q, k, v, o, lse, **kw)
    clean()
    args = (inp.cu_seqlens.tolist(), causal, D ** -0.5, cap, slopes)
    r = osh.forward(inp.q, inp.k, inp.v, *args)
    b = osh.backward(inp.q, inp.k, inp.v, inp.do, *args)
    # The bounds of the other cases; the scores reach |slope| N.
    e = score_error(inp.q, inp.k, D ** -0.5, cap, slopes.abs(), N, dtype)
    h = HALF if dtype == "bf16" else 2.0 ** -23
    inside("LSE", f64(lse).transpose(1, 0, 2).reshape(H, T), r.lse, e)
    inside("O", f64(o).reshape(T, H, D), r.o,
           (h * (1 + 2 * h) + 2 * e) * (r.o_abs + abs(r.o)) + h * abs(r.o))
    dq, dk, dv = (f64(x).reshape(y.shape) for x, y in zip(got, (b.dq, b.dk, b.dv)))
    tiny = e + D * 2.0 ** -23
    c = 2.0 ** -20 if cap else 0.0
    f = 2.0 ** -39 if dtype == "bf16" else 0.0
    inside("dV", dv, b.dv, (h + 2 * e) * b.dv_abs + h * abs(b.dv))
    for name, x, y, one, raw, full, delta in (("dQ", dq, b.dq, b.dq_one, b.dq_raw, b.dq_abs, b.dq_del),
                                              ("dK", dk, b.dk, b.dk_one, b.dk_raw, b.dk_abs, b.dk_del)):
        inside(name, x, y, f * one + c * raw + (2 * h + 4 * e) * full + (h + 2 * tiny) * delta + h * abs(y))


@pytest.mark.parametrize("page", [None, 64])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("D", [64, 128])
def test_negative_slopes_in_decode(D, cap, page):
    lengths, q_len, H, H_kv, most = [1, 129, 700, 2000], 3, 8, 2, 2000
    c = decode_case(21, dtype="bf16", lengths=lengths, q_len=q_len, H=H, H_kv=H_kv, D=D, page_size=page)
    if page is None:
        c.page_size = c.k_cache.shape[0] // len(lengths)
    slopes = torch.linspace(-0.4, 0.2, H)
    w = torch.zeros(len(lengths), H_kv, most, device="cuda")
    o, lse = fa.decode(c.q.cuda(), c.k_cache.cuda(), c.v_cache.cuda(), c.cache_seqlens.cuda(), q_len=q_len,
                       max_seqlen_k=most, page_size=c.page_size, softcap=cap or None,
                       block_table=None if page is None else c.block_table.cuda(),
                       alibi_slopes=slopes.cuda(), key_weights=w)
    clean()
    ro, rl, ra, rw = osh.decode(c.q, c.k_cache, c.v_cache, lengths, q_len=q_len, scale=D ** -0.5,
                                page_size=c.page_size, block_table=c.block_table, cap=cap, slopes=slopes,
                                slots=most)
    used = torch.isfinite(c.k_cache[:, 0, 0].float())
    e = score_error(c.q, c.k_cache[used], D ** -0.5, cap, slopes.abs(), most, "bf16")
    inside("LSE", f64(lse), rl, e)
    inside("O", f64(o), ro, (HALF + 2 * e) * ra + HALF * abs(ro))
    inside("weights", f64(w), rw, 2 * e * rw + 2.0 ** -22 * (1 + rw))


# ----------------------------------------------------------------- far offsets ---

def test_gradients_of_keys_past_2_31_elements():
    # 270 thousand tokens of 64 heads of 128, each seeing its last 40 keys: dK and dV of the
    # last tokens, whose queries all lie among the last ones too. Q and dO differ, so that a
    # row taken from elsewhere shows.
    N, H, D, window, m = 270_000, 64, 128, 40, 300
    g = torch.Generator("cuda").manual_seed(3)
    rnd = lambda h: torch.randn((1, N, h, D), generator=g, device="cuda", dtype=torch.bfloat16)
    q, do, k, v = rnd(H), rnd(H), rnd(1), rnd(1)
    begin = (torch.arange(N, device="cuda") - window + 1).clamp(min=0).int()[None]
    kw = dict(causal=True, softcap=30.0, key_begin=begin)
    o, lse = fa.fwd(q, k, v, **kw)
    _, dk, dv = fa.bwd(do, q, k, v, o, lse, **kw)
    clean()
    qq, gg, kk, vv = (x[0, N - m:].cpu() for x in (q, do, k, v))
    b = osh.backward(qq, kk, vv, gg, [0, m], True, D ** -0.5, 30.0, None,
                     np.maximum(0, np.arange(m) - window + 1))
    e = score_error(qq, kk, D ** -0.5, 30.0, None, m, "bf16")
    s = slice(window, m)   # from here on the queries see only keys among the last m
    inside("dV", f64(dv[0, N - m:])[s], b.dv[s], ((HALF + 2 * e) * b.dv_abs + HALF * abs(b.dv))[s])
    inside("dK", f64(dk[0, N - m:])[s], b.dk[s],
           (2.0 ** -39 * b.dk_one + 2.0 ** -20 * b.dk_raw + (2 * HALF + 4 * e) * b.dk_abs +
            (HALF + 2 * (e + D * 2.0 ** -23)) * b.dk_del + HALF * abs(b.dk))[s])
