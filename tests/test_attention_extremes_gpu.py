"""The attention operators where values are not finite or very large, and where
sizes and offsets leave the ordinary range."""

import math

import pytest
import torch

import input_dependent_short_b200 as dsc
from input_dependent_short_b200 import _lib

import attn_ref as ref
from test_attention_gpu import BF, F32, cu_of, gen, paged, qkv

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _device():
    if not torch.cuda.is_available():
        pytest.fail("needs a CUDA device")
    yield
    assert _lib.lib().dsc_check(torch.cuda.current_stream().cuda_stream) == _lib.DSC_OK


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 96])
def test_an_infinite_channel_leaves_the_others_as_precise(d, dtype):
    """One element infinite in every value row: infinite in o, while the other
    elements keep the bound that they have without it."""
    docs, Hq, Hkv = [300, 50, 128], 4, 2
    T = sum(docs)
    q, k, v = (t.clone() for t in qkv(T, Hq, Hkv, d, dtype, seed=120, gain=0.5))
    scale = 1 / math.sqrt(d)
    ro, bo, rl, bl = ref.attn_fwd(q, k, v, docs, scale, dtype)
    v[:, :, 5] = math.inf
    o, lse = dsc.dsc_fwd_attn_varlen(q, k, v, cu_of(docs))
    others = torch.arange(d, device="cuda") != 5
    assert torch.isposinf(o[:, :, 5]).all()
    ref.check("o", o[..., others], ro[..., others], bo[..., others])
    ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (3, 1), (7, 1), (4, 2)])
def test_a_bad_value_shows_in_every_row_that_sees_it(Hq, Hkv, dtype):
    """Odd groups and even ones, in both tiles of 128 that a block may own: a
    value row with one infinity or NaN shows in that element of all later rows,
    in no earlier row and no other document, and leaves the other elements their
    bound."""
    docs, d = [600, 50], 64
    T = sum(docs)
    q, k, v = (t.clone() for t in qkv(T, Hq, Hkv, d, dtype, seed=130, gain=0.5))
    cu, scale = cu_of(docs), 1 / math.sqrt(d)
    clean, _ = dsc.dsc_fwd_attn_varlen(q, k, v, cu)
    ro, bo, rl, bl = ref.attn_fwd(q, k, v, docs, scale, dtype)
    for at in (0, 40, 127, 128, 200, 255, 256, 300, 511, 599, 610):
        end = docs[0] if at < docs[0] else T
        keep = v[at].clone()
        for x in (math.inf, math.nan):
            v[at, :, 3] = x
            o, lse = dsc.dsc_fwd_attn_varlen(q, k, v, cu)
            v[at] = keep
            reached = torch.zeros(T, dtype=torch.bool, device="cuda")
            reached[at:end] = True
            assert not torch.isfinite(o[reached, :, 3]).any(), at
            assert torch.equal(o[~reached], clean[~reached]), at
            o[reached, :, 3] = clean[reached, :, 3]
            others = torch.arange(d, device="cuda") != 3
            ref.check(f"o {at}", o[..., others], ro[..., others], bo[..., others])
            ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(2, 1), (3, 3)])
@pytest.mark.parametrize("rise", [8, 12, 20, 28])
def test_large_values_do_not_overflow(rise, Hq, Hkv, dtype):
    """Values of 2^112 where the first 128 keys weigh 2^rise times as much as the
    later ones: the weighted sums stay below the number of keys times the values
    (600 x 2^113 < 2^123), however the running maximum moves."""
    n, d = 600, 64
    q = torch.zeros(n, Hq, d, device="cuda")
    k = torch.zeros(n, Hkv, d, device="cuda")
    q[:, :, 0] = 1.0
    k[:, :, 1:] = torch.randn(n, Hkv, d - 1, generator=gen(140), device="cuda")
    k[:128, :, 0] = rise * math.log(2.0)
    v = torch.randn(n, Hkv, d, generator=gen(141), device="cuda").clamp(-2, 2) * 2.0 ** 112
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    o, lse = dsc.dsc_fwd_attn_varlen(q, k, v, cu_of([n]), scale=1.0)
    ro, bo, rl, bl = ref.attn_fwd(q, k, v, [n], 1.0, dtype)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2), (6, 1)])
def test_scores_that_are_all_minus_infinity(Hq, Hkv, dtype):
    """Softmax over nothing but -infinity is 0 / 0: NaN, with lse -infinity, in the
    decode step as in the prompt; zeros are for sequences with nothing to read."""
    d, lens = 64, [1, 100, 0, 3000]
    kc, vc, table, sl = paged(lens, 16, Hkv, d, dtype, seed=150)
    kc[..., 2] = -kc[..., 2].abs() - 1
    q = torch.randn(4, Hq, d, generator=gen(151), device="cuda").to(dtype)
    clean = dsc.dsc_decode_attn(q, kc, vc, table, sl)
    q[:, 0, 2] = math.inf
    o, lse = dsc.dsc_decode_attn(q, kc, vc, table, sl)
    some = torch.tensor([0, 1, 3], device="cuda")
    assert torch.isnan(o[some, 0]).all() and torch.isneginf(lse[:, 0]).all()
    assert not o[2].any() and torch.isneginf(lse[2]).all()
    assert torch.equal(o[:, 1:], clean[0][:, 1:]) and torch.equal(lse[:, 1:], clean[1][:, 1:])

    # one key that is finite carries the row, wherever it lies
    kc[..., 2] = -math.inf
    for b in (0, 1, 3):
        pg = int(table[b, (lens[b] // 2) // 16])
        kc[pg, :, (lens[b] // 2) % 16, 2] = 0.5
    q[:, :, 2] = 1.0
    o, lse = dsc.dsc_decode_attn(q, kc, vc, table, sl)
    assert torch.isfinite(o).all() and torch.isfinite(lse[some]).all()
    for b in (0, 1, 3):
        at = lens[b] // 2
        want = vc[int(table[b, at // 16]), :, at % 16].repeat_interleave(Hq // Hkv, 0)
        assert torch.equal(o[b], want)          # a weight of one, exactly

    # the prompt
    x, k, v = (t.clone() for t in qkv(200, Hq, Hkv, d, dtype, seed=152))
    k[..., 2] = -k[..., 2].abs() - 1
    x[150, 0, 2] = math.inf
    o, lse = dsc.dsc_fwd_attn_varlen(x, k, v, cu_of([200]))
    assert torch.isnan(o[150, 0]).all() and torch.isneginf(lse[0, 150])
    assert torch.isfinite(o[torch.arange(200, device="cuda") != 150]).all()


def test_append_where_pages_times_heads_pass_2_31():
    """Pages of one token, so that a page's number times the heads passes 31 bits:
    every new row lies where the table says and where the decode step reads it."""
    Hq, Hkv, d, page = 16, 8, 8, 1
    torch.cuda.empty_cache()
    n_pages = 2 ** 31 // Hkv + 64               # 34 GB a cache
    kc, vc = (torch.empty(n_pages, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    first = n_pages - 48                        # page * heads >= 2^31 from here on
    assert first * Hkv > 2 ** 31
    new = [20, 1, 7]
    order = (first + torch.randperm(40, generator=gen(160), device="cuda")[:28]).to(torch.int32)
    table = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    t0 = 0
    for s, n in enumerate(new):
        table[s, :n] = order[t0:t0 + n]
        t0 += n
    for c in (kc, vc):
        c[:64] = 3.0
        c[first:] = 3.0
    q, k, v = qkv(28, Hq, Hkv, d, BF, seed=161)
    sl = torch.tensor(new, dtype=torch.int32, device="cuda")
    assert dsc.dsc_kv_append(None, k, v, kc, vc, table, sl, cu_seqlens=cu_of(new)) is None
    at = order.long()
    assert torch.equal(kc[at, :, 0], k) and torch.equal(vc[at, :, 0], v)
    rest = torch.ones(n_pages - first, dtype=torch.bool, device="cuda")
    rest[at - first] = False
    for c in (kc, vc):
        assert (c[:64] == 3).all() and (c[first:][rest] == 3).all()
    o, lse = dsc.dsc_decode_attn(q[:3].contiguous(), kc, vc, table, sl)
    ro, bo, rl, bl = ref.decode(q[:3], kc, vc, table, new, 1 / math.sqrt(d), BF)
    ref.check("o", o, ro, bo)
    ref.check("lse", lse, rl, bl)
    del kc, vc, c
    torch.cuda.empty_cache()


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("T,times", [(1000, 6), (4096, 30), (2 ** 20, 2 ** 18 + 5)])
def test_offsets_that_overlap_without_end_count_as_no_documents(T, times, dtype):
    """0, T, 0, T, ...: up to 2^18 documents of 2^20 rows, whose tiles pass 2^31.
    Zeros, at once, and nothing outside the outputs is touched.  (Few documents of
    few rows are a list that the bf16 kernels make themselves.)"""
    Hq, Hkv, d = 2, 1, 8
    q, k, v = qkv(T, Hq, Hkv, d, dtype, seed=170)
    cu = torch.tensor([0, T] * times, dtype=torch.int32, device="cuda")
    o, lse = dsc.dsc_fwd_attn_varlen(q, k, v, cu)
    assert not o.any() and torch.isneginf(lse).all()
    guard = torch.full((T + 2, (Hq + 2 * Hkv) * d), 7.0, dtype=dtype, device="cuda")
    h = guard[1:-1].unflatten(1, (Hq + 2 * Hkv, d))
    out = h[:, :Hq], h[:, Hq:Hq + Hkv], h[:, Hq + Hkv:]
    for g in dsc.dsc_bwd_attn_varlen(q, k, v, o, lse, o, cu, out=out):
        assert not g.any()
    assert (guard[0] == 7).all() and (guard[-1] == 7).all()
    # and the next call, with documents, is as ever
    n = min(T, 700)
    cu = cu_of([n // 3, n - n // 3])
    o, lse = dsc.dsc_fwd_attn_varlen(q[:n], k[:n], v[:n], cu)
    ro, bo, rl, bl = ref.attn_fwd(q[:n], k[:n], v[:n], [n // 3, n - n // 3], 1 / math.sqrt(d), dtype)
    ref.check("o", o, ro, bo)


def test_a_feed_whose_waits_run_out_hands_over_no_item():
    """The kernels' work feed with a wait that nothing ends (a few milliseconds):
    the reader and the drawing lane both stop, the time-out reaches the host and
    is cleared, and the next call is right."""
    L, s = _lib.lib(), torch.cuda.current_stream().cuda_stream
    assert L.dsc_check(s) == _lib.DSC_OK
    n0 = L.dsc_launch_count()
    assert L.dsc_selftest_attn_timeout(s) == _lib.DSC_OK
    assert L.dsc_launch_count() == n0 + 1
    assert L.dsc_check(s) == _lib.DSC_ERR_TIMEOUT
    assert L.dsc_check(s) == _lib.DSC_OK
    docs = [300, 77]
    q, k, v = qkv(377, 4, 2, 64, BF, seed=180)
    o, _ = dsc.dsc_fwd_attn_varlen(q, k, v, cu_of(docs))
    ro, bo, _, _ = ref.attn_fwd(q, k, v, docs, 0.125, BF)
    ref.check("o", o, ro, bo)


def without_the_rounding_of_o(bound, q, k, v, do, scale):
    """attn_ref's bound of a document's dq less what it allows for a D = do . o
    that comes from a rounded o: D as an fp32 sum over the probabilities."""
    n, Hq, _ = q.shape
    u, g = ref.U[BF], Hq // k.shape[1]
    seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
    far = (torch.arange(n, device="cuda") >= 128).double()[:, None]
    out = bound.clone()
    for h in range(Hq):
        qq, kk, vv, gg = q[:, h].double(), k[:, h // g].double(), v[:, h // g].double(), do[:, h].double()
        _, _, p, _, eP = ref._probs(qq, kk, scale, seen)
        mean = (p * (gg.abs() @ vv.abs().T)).sum(1, keepdim=True)
        out[:, h] -= (1 + u) * scale * ((p * ((2 * u + eP) * mean * far)) @ kk.abs())
    return out


@pytest.mark.parametrize("d", [64, 96, 128])
@pytest.mark.parametrize("n", [129, 256, 257, 385, 700])
def test_dq_of_rows_that_one_key_carries(n, d):
    """The first key takes all but 2^-8 or less of every row, so dP - D is small
    beside D: o rounds to 1 - 2^-9 +- 2^-9 and a D that came from it would be off
    by up to 2^-9, five times the bound."""
    Hq, Hkv, scale = 2, 1, 1 / math.sqrt(d)
    q, k, v = (0.3 * torch.randn(n, h, d, generator=gen(190 + i), device="cuda") for i, h in enumerate((Hq, Hkv, Hkv)))
    q[..., 0], k[..., 0] = 1.0, 0.0
    k[0, :, 0] = math.log(n * 2.0 ** 8) / scale
    v[0] = 1.0
    q, k, v = q.to(BF), k.to(BF), v.to(BF)
    do = torch.ones(n, Hq, d, dtype=BF, device="cuda")
    cu = cu_of([n])
    o, lse = dsc.dsc_fwd_attn_varlen(q, k, v, cu)
    got = dsc.dsc_bwd_attn_varlen(q, k, v, o, lse, do, cu)
    want, bound = ref.attn_bwd(q, k, v, do, [n], scale, BF)
    bound[0] = without_the_rounding_of_o(bound[0], q, k, v, do, scale)
    for name, g, w, b in zip(("dq", "dk", "dv"), got, want, bound):
        ref.check(name, g, w, b)


@pytest.mark.parametrize("docs,Hq,Hkv,d", [([700, 129, 300], 4, 2, 128), ([1500], 3, 3, 64), ([257, 640], 7, 1, 96)], ids=str)
def test_dq_is_as_near_as_its_own_roundings_leave_it(docs, Hq, Hkv, d):
    """Sharp rows (scores of a standard deviation of 4): dq within the bound that
    counts the rounding of dS and of the result alone, and in the mean square no
    further off than these two roundings, each uniform over a step (2^-8 / sqrt 3
    relative at most)."""
    T, scale, t0 = sum(docs), 1 / math.sqrt(d), 0
    q, k, v = qkv(T, Hq, Hkv, d, BF, seed=200, gain=4.0)
    do = torch.randn(T, Hq, d, generator=gen(201), device="cuda").to(BF)
    cu = cu_of(docs)
    o, lse = dsc.dsc_fwd_attn_varlen(q, k, v, cu)
    dq = dsc.dsc_bwd_attn_varlen(q, k, v, o, lse, do, cu)[0]
    want, bound = ref.attn_bwd(q, k, v, do, docs, scale, BF)
    for n in docs:
        r = slice(t0, t0 + n)
        ref.check("dq", dq[r], want[0][r], without_the_rounding_of_o(bound[0][r], q[r], k[r], v[r], do[r], scale))
        t0 += n
    err = ((dq.double() - want[0]).norm() / want[0].norm()).item()
    print(f"dq: {err:.5f} of its norm")
    assert err <= math.sqrt(2) * 2.0 ** -8 / math.sqrt(3)
