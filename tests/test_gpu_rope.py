"""Rotary positions on the GPU against the fp64 oracle.

Per value y of a head, from the arithmetic (u = 2^-24), with h the length of its
pair after norm and magnitude (|y| itself where nothing turns):
  * y is rounded to bf16: 2^-8 |y|;
  * the turn goes to fp32 with 2^-26 of a turn, 2 pi 2^-26 < 2^-23 radians, and
    the sine and cosine to fp32 within 2 units in the last place, 2^-23; times
    the magnitude, the product and the sum: 3 u more. Less than 2^-21 h;
  * a norm: a sum of squares in a chain of 16 and 4 additions, the division,
    eps, the root (2 units) and two products: less than 28 u, half of it after
    the root but for the last ones. Less than 2^-19 h.
So |got - want| <= 2^-8 |want| + 2^-18 h.
"""
import numpy as np
import pytest
import torch

from oracle import paged
from oracle.moe import bf16_bits_to_f64
from tests._util import bits16

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
KINDS = dict(plain=0, linear=1, bands=2, ramp=3)


def _bf(gen, *shape, std=1.0):
    return (torch.randn(shape, generator=gen) * std).to(torch.bfloat16)


def _i32(v):
    return torch.tensor([int(x) for x in v], dtype=torch.int32, device=DEV)


def make_spec(m, D, rot, pairs=False, norm=0, gains=True, offset=0.0, scaling="plain", base=1e4, factor=1.0, original=0,
              eps=1e-6, seed=9):
    """A spec and what the oracle needs of it."""
    gen = torch.Generator().manual_seed(seed)
    g = [(1 - offset + 0.3 * torch.randn(D, generator=gen)).to(torch.bfloat16) for _ in range(2)] if gains else [None] * 2
    table = m.rope_table(rot, base, KINDS[scaling], factor, original, device=DEV) if rot else None
    spec = m.rope_spec(table, m.ROPE_PAIRS if pairs else m.ROPE_HALF, norm, *[None if x is None else x.to(DEV) for x in g],
                       eps=eps, gain_offset=offset)
    w, mag = paged.frequencies(rot, base, scaling, factor, original) if rot else (np.zeros(0), 1.0)
    g = [None if x is None else bf16_bits_to_f64(bits16(x)) for x in g]

    def oracle(x, positions, key=False):
        """fp64 heads as the spec makes them, and the length h of each value's pair."""
        y = bf16_bits_to_f64(bits16(x))
        if norm & (2 if key else 1):
            y = paged.normed(y, g[key], eps, offset)
        z = paged.rotated(y, positions, w, pairs, mag) if rot else y
        h = np.abs(z)
        if rot:
            one, two = (slice(0, rot, 2), slice(1, rot, 2)) if pairs else (slice(0, rot // 2), slice(rot // 2, rot))
            h[..., one] = h[..., two] = np.hypot(z[..., one], z[..., two])
        return z, h

    return spec, oracle


def check(got, want, h):
    got = got.double().cpu().numpy()
    err, tol = np.abs(got - want), 2.0 ** -8 * np.abs(want) + 2.0 ** -18 * h
    assert np.isfinite(got).all() and (err <= tol).all(), (float((err - tol).max()), np.argwhere(err > tol)[:4])


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,norm,scaling", [
    (1, 16, 2, 256, 64, 3, "plain"), (1, 1, 0, 16, 16, 0, "plain"), (3, 0, 5, 64, 32, 2, "linear"),
    (77, 3, 1, 80, 80, 1, "bands"), (50, 7, 7, 48, 48, 3, "ramp"), (130, 40, 8, 128, 128, 0, "ramp"),
    (33, 5, 2, 192, 112, 3, "plain"), (9, 4, 1, 240, 16, 3, "bands"), (600, 16, 2, 256, 256, 3, "linear"),
    (4000, 6, 3, 32, 32, 3, "plain"), (2, 2, 2, 96, 0, 3, "plain"), (1500, 16, 4, 16, 16, 3, "plain")])
def test_rope_is_the_oracles(moelib, cuda_dev, T, Hq, Hk, D, rot, norm, scaling, pairs):
    m = moelib
    spec, oracle = make_spec(m, D, rot, pairs, norm, True, 1.0 if T % 2 else 0.0, scaling, 1e4, 8.0, 4096)
    gen = torch.Generator().manual_seed(T)
    q, k = _bf(gen, T, Hq, D), _bf(gen, T, Hk, D, std=3.0)
    pos = torch.randint(0, 1 << 20, (T,), generator=gen).tolist()
    qo, ko = (torch.full(x.shape, float("nan"), dtype=torch.bfloat16, device=DEV) for x in (q, k))
    m.rope(m.rope_shape(T, Hq, Hk, D), spec, q.to(DEV) if Hq else None, k.to(DEV) if Hk else None,
           _i32(pos) if rot else None, qo if Hq else None, ko if Hk else None)
    if Hq:
        check(qo, *oracle(q, pos))
    if Hk:
        check(ko, *oracle(k, pos, True))


@pytest.mark.parametrize("T", [5, 700])
def test_strides_and_in_place(moelib, cuda_dev, T):
    """q and k as column ranges of one projection, turned in place; what lies between and around them stays."""
    m = moelib
    spec, oracle = make_spec(m, 128, 64, norm=3)
    gen = torch.Generator().manual_seed(2)
    x = _bf(gen, T + 1, 13 * 128)
    y = x.to(DEV)
    q, k = y[:T, :8 * 128].view(T, 8, 128), y[:T, 9 * 128:11 * 128].view(T, 2, 128)
    pos = list(range(7, 7 + T))
    sh = m.rope_shape(T, 8, 2, 128, 13 * 128, 13 * 128, 13 * 128, 13 * 128)
    m.rope(sh, spec, q, k, _i32(pos), q, k)
    check(q, *oracle(x[:T, :1024].view(T, 8, 128), pos))
    check(k, *oracle(x[:T, 1152:1408].view(T, 2, 128), pos, True))
    rest = torch.ones(T + 1, 13 * 128, dtype=torch.bool)
    rest[:T, :1024] = rest[:T, 1152:1408] = False
    assert torch.equal(y.cpu()[rest], x[rest])
    # packed outputs give the same bits
    qo, ko = torch.empty(T, 8, 128, dtype=torch.bfloat16, device=DEV), torch.empty(T, 2, 128, dtype=torch.bfloat16, device=DEV)
    z = x.to(DEV)
    m.rope(m.rope_shape(T, 8, 2, 128, 13 * 128, 13 * 128), spec, z[:T, :1024].view(T, 8, 128),
           z[:T, 1152:1408].view(T, 2, 128), _i32(pos), qo, ko)
    assert torch.equal(qo, q) and torch.equal(ko, k)


@pytest.mark.parametrize("pairs", [False, True])
def test_far_and_negative_positions(moelib, cuda_dev, pairs):
    """Positions at the ends of int32 are as exact as near ones: the table's own rounding, 2^-54 of a turn, is 2^-23 at
    2^31, 2^-20 radians of h (within the 2^-18)."""
    pos = [2 ** 31 - 1, -2 ** 31, -1, 0, 1 << 30, -12345, 99999999]
    spec, oracle = make_spec(moelib, 64, 64, pairs, base=1e6)
    q = _bf(torch.Generator().manual_seed(3), len(pos), 3, 64)
    qo = torch.empty_like(q, device=DEV)
    moelib.rope(moelib.rope_shape(len(pos), 3, 0, 64), spec, q.to(DEV), None, _i32(pos), qo, None)
    check(qo, *oracle(q, pos))


def test_gains_left_out_and_norm_of_one_side(moelib, cuda_dev):
    for norm in (0, 1, 2, 3):
        spec, oracle = make_spec(moelib, 128, 32, norm=norm, gains=False, offset=5.0)
        gen = torch.Generator().manual_seed(4)
        q, k, pos = _bf(gen, 20, 3, 128), _bf(gen, 20, 2, 128), list(range(20))
        qo, ko = torch.empty_like(q, device=DEV), torch.empty_like(k, device=DEV)
        moelib.rope(moelib.rope_shape(20, 3, 2, 128), spec, q.to(DEV), k.to(DEV), _i32(pos), qo, ko)
        check(qo, *oracle(q, pos))
        check(ko, *oracle(k, pos, True))


@pytest.mark.parametrize("D", [16, 64, 256])
def test_norm_of_any_finite_head(moelib, cuda_dev, D):
    """Heads of bf16's largest values, whose squares pass fp32, of its smallest, and of zeros; eps beside them."""
    spec, oracle = make_spec(moelib, D, 16, norm=3, eps=1e-6)
    gen = torch.Generator().manual_seed(5)
    sizes = torch.tensor([3e38, 1e30, 2e19, 1e18, 1.0, 1e-3, 1e-20, 1e-38, 0.0])
    u = torch.randn(len(sizes), 2, D, generator=gen).clamp(-1, 1)
    q = (u * sizes[:, None, None]).to(torch.bfloat16)
    q[1, 0, 0] = 3.38e38  # one large value among smaller ones
    pos = list(range(len(sizes)))
    qo = torch.empty_like(q, device=DEV)
    moelib.rope(moelib.rope_shape(len(sizes), 2, 0, D), spec, q.to(DEV), None, _i32(pos), qo, None)
    want, h = oracle(q, pos)
    h = h + 2.0 ** -115  # (what fp32 and bf16 flush or round below their normal numbers)
    check(qo, want, h)


def test_a_head_that_is_not_finite_stays_alone(moelib, cuda_dev):
    spec, _ = make_spec(moelib, 128, 64, norm=3)
    gen = torch.Generator().manual_seed(6)
    q = _bf(gen, 40, 8, 128).to(DEV)
    sh, pos = moelib.rope_shape(40, 8, 0, 128), _i32(range(40))
    a, b = torch.empty_like(q), torch.empty_like(q)
    moelib.rope(sh, spec, q, None, pos, a, None)
    q[7, 3, 100], q[20, 0, 5], q[39, 7, 127] = float("nan"), float("inf"), float("-inf")
    moelib.rope(sh, spec, q, None, pos, b, None)
    other = torch.ones(40, 8, dtype=torch.bool)
    other[7, 3] = other[20, 0] = other[39, 7] = False
    assert torch.equal(a[other.to(DEV)], b[other.to(DEV)])
    assert all(torch.isnan(b[i, j]).any() for i, j in ((7, 3), (20, 0), (39, 7)))


def test_refusals_of_the_binding(moelib, cuda_dev):
    m = moelib
    q = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    pos, spec = _i32(range(4)), make_spec(m, 64, 16, norm=1)[0]
    sh = m.rope_shape(4, 2, 0, 64)
    for text, call in [("q is torch.float16", lambda: m.rope(sh, spec, q.half(), None, pos, q, None)),
                       ("q has shape", lambda: m.rope(sh, spec, q[:3], None, pos, q, None)),
                       ("q_out has strides", lambda: m.rope(sh, spec, q, None, pos, q.transpose(0, 1).contiguous().transpose(0, 1), None)),
                       ("positions is torch.int64", lambda: m.rope(sh, spec, q, None, pos.long(), q, None)),
                       ("positions is on cpu", lambda: m.rope(sh, spec, q, None, pos.cpu(), q, None)),
                       ("k is torch.float32", lambda: m.rope(m.rope_shape(4, 2, 2, 64), spec, q, q.float(), pos, q, q)),
                       ("the spec's tensors are for heads of 64", lambda: m.rope(m.rope_shape(4, 1, 0, 128), spec, q.view(4, 1, 128), None, pos, q.view(4, 1, 128), None)),
                       ("invalid argument", lambda: m.rope(sh, spec, q, None, None, q, None))]:
        with pytest.raises(m.MoeError, match=text):
            call()


def test_rope_in_a_graph_follows_its_inputs(moelib, cuda_dev):
    m = moelib
    spec, oracle = make_spec(m, 256, 64, norm=3)
    gen = torch.Generator().manual_seed(8)
    x = [_bf(gen, 9, 4, 256) for _ in range(2)]
    q, pos, qo = x[0].to(DEV), _i32(range(9)), torch.empty(9, 4, 256, dtype=torch.bfloat16, device=DEV)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        m.rope(m.rope_shape(9, 4, 0, 256), spec, q, None, pos, qo, None)
    q.copy_(x[1]), pos.add_(1000)
    g.replay()
    check(qo, *oracle(x[1], list(range(1000, 1009))))
    m.rope(m.rope_shape(0, 4, 0, 256), spec, q[:0], None, pos[:0], qo[:0], None)  # no tokens


@pytest.mark.parametrize("D,eps,gain,sizes", [
    (64, 1e37, 1.0, [1e19, 5e18, 3e19, 1.0, 0.0]),       # eps beside squares whose sum passes fp32
    (16, 3.35e38, 1.0, [4e18, 4.2e18, 1e10, 3e38]),      # a mean that passes fp32 with eps, not without
    (128, 1e-6, 1e37, [1e-5, 1e-3, 1e-8, 0.0]),          # gains that pass fp32 with a small head's factor
    (128, 1e-6, 1e-30, [1e12, 1e16, 1e18, 3e38])])       # ... and fall below it with a large one's
def test_norm_with_eps_and_gains_near_the_ends_of_fp32(moelib, cuda_dev, D, eps, gain, sizes):
    """Every finite eps and gain. (Where values, gains or results are below fp32's normal numbers, 2^-126, the factor
    may lose that much of them: 2^-120.)"""
    m = moelib
    gen = torch.Generator().manual_seed(11)
    g = ((1 + 0.2 * torch.rand(D, generator=gen)) * gain).to(torch.bfloat16)
    spec = m.rope_spec(None, norm=m.ROPE_NORM_Q, q_gain=g.to(DEV), eps=eps)
    u = torch.randn(len(sizes), 3, D, generator=gen).clamp(-1, 1)
    q = (u * torch.tensor(sizes)[:, None, None]).to(torch.bfloat16)
    q[:, 0, 3] = 0.0
    qo = torch.empty_like(q, device=DEV)
    m.rope(m.rope_shape(len(sizes), 3, 0, D), spec, q.to(DEV), None, None, qo, None)
    want = paged.normed(bf16_bits_to_f64(bits16(q)), bf16_bits_to_f64(bits16(g)), float(np.float32(eps)))
    check(qo, want, np.abs(want) + 2.0 ** -102)
