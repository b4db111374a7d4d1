"""Rotary positions with several axes on the GPU against the float64 oracle.

Tolerance.  cos and sin are float32 of an angle that is exact to 2^-25 turns
(float32 of the 32-bit fraction) and come from sincospif (2 ulp): each is off by
at most 2 pi 2^-25 + 2^-22 < 2^-21.  Two products and a sum in float32 add less
than 2^-22 of |x1| + |x2|.  So y before its rounding is within 2^-20 (|x1| + |x2|),
and the rounding to bfloat16 adds 2^-8 |y| (half a step)."""
import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import attn_fwd_status, attn_rope, attn_rope_axes, attn_rope_bwd, attn_rope_table
from exact_attention_attn_gb300.workloads import to_f64
from oracle import serving as S

pytestmark = pytest.mark.gpu


def _check(y, x, pos, inv, axis, adjacent, backward=False):
    want = S.rope(to_f64(x), pos.cpu().numpy(), inv, axis, adjacent, backward)
    rot, xs = 2 * len(inv), np.abs(to_f64(x))
    pair = xs.copy()
    a, b = (xs[..., 0:rot:2], xs[..., 1:rot:2]) if adjacent else (xs[..., :rot // 2], xs[..., rot // 2:rot])
    both = a + b
    pair[..., :rot] = np.repeat(both, 2, -1) if adjacent else np.concatenate([both, both], -1)
    got = to_f64(y)
    tol = 2.0 ** -20 * pair + 2.0 ** -8 * np.abs(want)
    tol[..., rot:] = 0.0
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], want[bad][:4])


def _inputs(B, Hq, Hkv, N, D, axes, span, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Hq, N, D), generator=g).to(torch.bfloat16).cuda()
    k = torch.randn((B, Hkv, N, D), generator=g).to(torch.bfloat16).cuda()
    pos = torch.randint(0, span, (axes, B, N), generator=g, dtype=torch.int32).cuda()
    return q, k, pos


CASES = [
    # B, Hq, Hkv, N, D, rot, sections, interleave, adjacent, span
    (1, 1, 1, 1, 64, 64, (32,), False, False, 10),
    (2, 4, 2, 17, 64, 16, (8,), False, True, 5000),
    (1, 32, 8, 33, 128, 128, (24, 20, 20), False, False, 1000000),
    (3, 3, 1, 5, 192, 96, (16, 0, 32), True, True, 100000),
    (1, 5, 5, 700, 128, 112, (20, 36), True, False, 1 << 31),
    (1, 2, 1, 9, 1024, 1024, (100, 200, 212), False, True, 70000),
    (2, 1, 1, 1300, 256, 256, (128,), False, False, 1 << 20),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("backward", [False, True])
def test_rope_matches_oracle(case, backward):
    B, Hq, Hkv, N, D, rot, sections, interleave, adjacent, span = case
    q, k, pos = _inputs(B, Hq, Hkv, N, D, len(sections), span, seed=D + N)
    inv = [10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)]
    table = attn_rope_table(rot, sections, interleave=interleave)
    axis = attn_rope_axes(sections, interleave)
    turn = attn_rope_bwd if backward else attn_rope
    oq, ok = turn(q, k, pos, table, adjacent=adjacent)
    torch.cuda.synchronize()
    assert attn_fwd_status() == 0
    _check(oq, q, pos, inv, axis, adjacent, backward)
    _check(ok, k, pos, inv, axis, adjacent, backward)


def test_rope_strides_in_place_and_one_tensor():
    B, N, H, D = 2, 19, 3, 128
    g = torch.Generator().manual_seed(4)
    fused = torch.randn((B, N, 3 * H, D), generator=g).to(torch.bfloat16).cuda()  # q, k, v heads of one projection
    before = fused.clone()
    q, k = (fused[:, :, i * H:(i + 1) * H].transpose(1, 2) for i in (0, 1))
    pos = torch.randint(0, 900, (1, 1, N), generator=g, dtype=torch.int32).cuda().expand(2, B, N)  # one row for both axes
    table = attn_rope_table(64, [10, 22], base=500.0)
    inv, axis = [500.0 ** (-2.0 * i / 64) for i in range(32)], attn_rope_axes([10, 22])
    ref_q, ref_k = attn_rope(q, k, pos, table)
    assert ref_q.shape == q.shape
    _check(ref_q, q, pos, inv, axis, False)
    only, none = attn_rope(q, None, pos, table)
    assert none is None and torch.equal(only, ref_q)
    attn_rope(q, k, pos, table, out_q=q, out_k=k)
    torch.cuda.synchronize()
    assert torch.equal(q, ref_q) and torch.equal(k, ref_k)
    assert torch.equal(fused[:, :, 2 * H:], before[:, :, 2 * H:])  # v's heads untouched
    with pytest.raises(ValueError, match="expanded"):
        attn_rope(ref_q, None, pos, table, out_q=torch.empty(1, 1, 1, D, dtype=torch.bfloat16, device="cuda").expand(B, H, N, D))


def test_rope_negative_and_far_positions_and_special_values():
    D = 64
    pos = torch.tensor([[[-5, -(2 ** 31), 2 ** 31 - 1, 0]]], dtype=torch.int32).cuda()
    inv = [1.0, 0.3, 6.5, -0.25] + [1e-3] * 28
    table = attn_rope_table(D, inv_freq=inv)
    q = torch.randn((1, 2, 4, D), generator=torch.Generator().manual_seed(0)).to(torch.bfloat16).cuda()
    o, _ = attn_rope(q, None, pos, table)
    _check(o, q, pos, inv, [0] * 32, False)
    assert torch.equal(o[:, :, 3], q[:, :, 3])  # position 0: cos 1, sin 0
    q[0, 0, 0, 0], q[0, 1, 1, 40] = float("inf"), float("nan")
    o, _ = attn_rope(q, None, pos, table)
    bad = ~torch.isfinite(o[0])
    want = torch.zeros_like(bad)
    want[0, 0, [0, 32]] = True
    want[1, 1, [8, 40]] = True
    assert torch.equal(bad.cpu(), want.cpu())


def test_rope_gradient_by_differences():
    # <w, rope(x + d) - rope(x - d)> against <rope_bwd(w), 2 d>: every value a small power of two, so that the only
    # errors are the outputs' roundings (2^-8 of 2 |x| per element, 64 x 6 elements of weight at most 1)
    g = torch.Generator().manual_seed(9)
    B, H, N, D = 1, 2, 3, 64
    x, w, d = (torch.randn((B, H, N, D), generator=g).to(torch.bfloat16).cuda() for _ in range(3))
    pos = torch.randint(0, 50, (1, B, N), generator=g, dtype=torch.int32).cuda()
    table = attn_rope_table(D)
    up, dn = (x + d).to(torch.bfloat16), (x - d).to(torch.bfloat16)
    yu, yd = attn_rope(up, dn, pos, table)
    dx, _ = attn_rope_bwd(w, None, pos, table)
    lhs = (w.double() * (yu.double() - yd.double())).sum()
    rhs = (dx.double() * (up.double() - dn.double())).sum()
    tol = 2.0 ** -8 * ((w.double().abs() * (yu.double().abs() + yd.double().abs())).sum()
                       + (dx.double().abs() * (up.double() - dn.double()).abs()).sum())
    assert abs(lhs - rhs) <= tol and abs(lhs) > 0


def test_rope_bad_axis_is_reported():
    q, _, pos = _inputs(1, 2, 1, 4, 64, 1, 100, 3)
    table = attn_rope_table(64, [16, 16])  # two axes, positions of one
    attn_rope(q, None, pos, table)
    assert attn_fwd_status() == -7 and attn_fwd_status() == 0
    o, _ = attn_rope(q, None, pos, attn_rope_table(64))
    assert attn_fwd_status() == 0


def test_rope_empty():
    table = attn_rope_table(64)
    for shape in ((0, 2, 3, 64), (2, 2, 0, 64)):
        q = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        o, _ = attn_rope(q, None, torch.empty((1, shape[0], shape[2]), dtype=torch.int32, device="cuda"), table)
        assert o.shape == shape


def test_rope_eight_axes_and_sections_of_nothing():
    sections = (3, 0, 5, 1, 7, 0, 8, 8)
    q, k, pos = _inputs(1, 3, 2, 37, 64, 8, 50000, seed=12)
    inv = [10000.0 ** (-2.0 * i / 64) for i in range(32)]
    for interleave in (False, True):
        axis = attn_rope_axes(sections, interleave)
        oq, ok = attn_rope(q, k, pos, attn_rope_table(64, sections, interleave=interleave))
        _check(oq, q, pos, inv, axis, False)
        _check(ok, k, pos, inv, axis, False)
    assert attn_fwd_status() == 0
