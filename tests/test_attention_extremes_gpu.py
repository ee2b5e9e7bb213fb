"""The attention operators where values are not finite or very large, and where
sizes and offsets leave the ordinary range."""

import math

import pytest
import torch

import input_dependent_short_b200 as dsc
from input_dependent_short_b200 import _lib

import attn_ref as ref
from test_attention_gpu import BF, F32, cu_of, gen, qkv

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
