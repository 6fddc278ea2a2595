"""Norm and rotation of query and key heads against the formula in 64 bits.

Tolerance: one rounding to bf16 (2^-8 of the value) and fp32 arithmetic on
the terms of the value's sum: the norm's factor (sum of up to 256 squares,
rsqrt, two products) and the rotation (sine and cosine of an angle rounded to
fp32 after reduction to [-pi, pi], two products, one sum) stay below 2^-18 of
the sum of the terms' sizes.
"""
import pytest
import torch

from tests import cache_ref as R

pytestmark = pytest.mark.gpu

S = None
EPS = 1e-6


@pytest.fixture(autouse=True)
def _lib():
    global S
    from lossless_kv_cache_bf16_gb300 import splitzip

    S = splitzip


def check(got, want, size):
    got = got.double().cpu()
    err = (got - want).abs()
    tol = 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -18 * size + 1e-30
    assert bool((err <= tol).all()), float((err - tol).max())


def inputs(tokens, hq, hk, dim, rot, seed, far=100000):
    g = R.gen(seed)
    q, k = R.normal_bf16(g, tokens, hq, dim, scale=3), R.normal_bf16(g, tokens, hk, dim)
    wq, wk = ((1 + 0.3 * torch.randn(dim, generator=g)).to(torch.bfloat16) for _ in range(2))
    freq = (10000.0 ** (-torch.arange(rot // 2) * 2.0 / max(rot, 1))).float()
    pos = torch.randint(0, far, (tokens,), generator=g, dtype=torch.int32)
    return q, k, wq, wk, freq, pos


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,hq,hk,dim,rot", [
    (1, 1, 1, 64, 64), (1, 32, 8, 128, 128), (3, 7, 1, 128, 48), (65, 28, 4, 128, 64), (17, 5, 3, 64, 16),
    (9, 12, 2, 256, 256), (33, 4, 4, 256, 96), (700, 8, 2, 128, 128), (5, 3, 2, 128, 0)])
def test_matches_the_formula(tokens, hq, hk, dim, rot, interleaved):
    q, k, wq, wk, freq, pos = inputs(tokens, hq, hk, dim, rot, seed=tokens + dim + rot)
    qo, ko = torch.empty_like(q.cuda()), torch.empty_like(k.cuda())
    S.sz_qk_norm_rope(q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), EPS, freq.cuda(), pos.cuda(), qo, ko, interleaved=interleaved)
    check(qo, *R.norm_rope(q, wq, EPS, freq, pos, interleaved))
    check(ko, *R.norm_rope(k, wk, EPS, freq, pos, interleaved))


@pytest.mark.parametrize("interleaved", [False, True])
def test_extreme_positions(interleaved):
    q, k, wq, wk, freq, pos = inputs(6, 2, 1, 128, 128, seed=4)
    pos[:] = torch.tensor([0, -1, 2 ** 31 - 1, -2 ** 31, 16777217, 999999937])
    qo, ko = torch.empty_like(q.cuda()), torch.empty_like(k.cuda())
    S.sz_qk_norm_rope(q.cuda(), k.cuda(), wq.cuda(), wk.cuda(), EPS, freq.cuda(), pos.cuda(), qo, ko, interleaved=interleaved)
    check(qo, *R.norm_rope(q, wq, EPS, freq, pos, interleaved))
    check(ko, *R.norm_rope(k, wk, EPS, freq, pos, interleaved))


@pytest.mark.parametrize("which", ["q", "k", "none"])
@pytest.mark.parametrize("hq,hk", [(4, 2), (5, 3)])     # 3 and 5: rows of both tensors in one warp
def test_norm_is_optional(which, hq, hk):
    q, k, wq, wk, freq, pos = inputs(11, hq, hk, 128, 64, seed=6)
    wq, wk = wq if which == "q" else None, wk if which == "k" else None
    qo, ko = torch.empty_like(q.cuda()), torch.empty_like(k.cuda())
    S.sz_qk_norm_rope(q.cuda(), k.cuda(), None if wq is None else wq.cuda(), None if wk is None else wk.cuda(), EPS,
                      freq.cuda(), pos.cuda(), qo, ko)
    check(qo, *R.norm_rope(q, wq, EPS, freq, pos, False))
    check(ko, *R.norm_rope(k, wk, EPS, freq, pos, False))


@pytest.mark.parametrize("layout", ["packed", "transposed", "odd offset", "odd head stride", "in place"])
def test_strides_alignment_and_in_place(layout):
    tokens, hq, hk, dim = 19, 6, 2, 128
    q, k, wq, wk, freq, pos = inputs(tokens, hq, hk, dim, 128, seed=8)
    if layout == "transposed":
        qd, kd = (x.cuda().transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k))
        qo, ko = torch.empty_strided(q.shape, qd.stride(), dtype=q.dtype, device="cuda"), torch.empty_like(k.cuda())
    else:
        row = 1 if layout == "odd offset" else 0
        width = dim + (3 if layout == "odd head stride" else 0)
        flat = torch.zeros(row + tokens * (hq + hk) * width, dtype=torch.bfloat16, device="cuda")
        qkv = flat[row:].view(tokens, hq + hk, width)[..., :dim]
        qkv[:, :hq], qkv[:, hq:] = q.cuda(), k.cuda()
        qd, kd = qkv[:, :hq], qkv[:, hq:]
        qo, ko = (qd, kd) if layout == "in place" else (torch.empty_like(q.cuda()), torch.empty_like(k.cuda()))
    S.sz_qk_norm_rope(qd, kd, wq.cuda(), wk.cuda(), EPS, freq.cuda(), pos.cuda(), qo, ko)
    check(qo, *R.norm_rope(q, wq, EPS, freq, pos, False))
    check(ko, *R.norm_rope(k, wk, EPS, freq, pos, False))


def test_zero_rows_nan_and_no_heads():
    q, k, wq, wk, freq, pos = inputs(4, 3, 2, 64, 32, seed=9)
    q[1] = 0
    q[2, 1, 5] = float("nan")
    qo = torch.empty_like(q.cuda())
    none = torch.empty(4, 0, 64, dtype=torch.bfloat16, device="cuda")
    S.sz_qk_norm_rope(q.cuda(), none, wq.cuda(), None, EPS, freq.cuda(), pos.cuda(), qo, none)
    assert bool((qo[1] == 0).all())
    assert bool(torch.isnan(qo[2, 1]).all()) and not bool(torch.isnan(qo[2, 0]).any())
    ok = [0, 1, 3]
    want, size = R.norm_rope(q, wq, EPS, freq, pos, False)
    check(qo[ok], want[ok], size[ok])
