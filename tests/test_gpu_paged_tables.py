"""Entries of the paged cache's tables that break the rules: reported, and nothing out of the arrays is touched."""
import numpy as np
import pytest
import torch

from oracle import paged
from tests._util import bits16
from tests.test_gpu_paged import DEV, Paged, _i32, _packed, _rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("start,path", [
    (10, [-2, -1, 0]), (0, [-100, -99, 0]), (0, [-2 ** 31, -2 ** 31 + 1, -2 ** 31 + 2]), (31, [-1, 0, 0]), (30, [0, 0, 1]),
    (10, [3, 1, 2]), (10, [5, 0, 1]), (32, [0, 1, 2]), (29, [0, 1, 3])])
def test_keep_refuses_entries_behind_their_place(moelib, cuda_dev, start, path):
    """Entries that increase after a bad one, but lie before the place they move to: of the last sequence, whose row of
    the table ends the array."""
    m = moelib
    p = Paged(m, [32, 32], 2, 64, 16, seed=42)
    out, st = _i32([-5, -5]), torch.zeros(1, dtype=torch.int32, device=DEV)
    m.paged_keep(p.shape(0, 2), p.gpu, _i32([20, start]), _i32([3, 3]), _i32([[0, 2, 7], path]), lens_out=out, status=st)
    assert m.status_read(st) == m.MOE_ERR_INVALID_ARG and out.tolist() == [23, -5]
    for bits, gpu in ((p.k, p.gpu.k), (p.v, p.gpu.v)):
        paged.keep(bits, p.tables, 16, [20, 0], [[0, 2, 7], []], [3, 0])
        assert np.array_equal(bits16(gpu), bits)


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("news", [[1, 1], [40, 40]])
def test_every_negative_page_is_reported(moelib, cuda_dev, news, D, page):
    """On single blocks and on pairs, in the context's first, a middle and its last page."""
    m = moelib
    p = Paged(m, [700, 300], 2, D, page, seed=91)
    T = sum(news)
    q = _rand(torch.Generator().manual_seed(92), T, 8, D).to(DEV)
    good = p.attend(q, news)
    sh = p.shape(T, 8)
    ws = m.paged_alloc_workspace(sh, DEV)
    for bad in (-2, -1, -3, -2 ** 31, -2 ** 31 + 1):
        for j in (0, (699 // page) // 2, 699 // page):
            old = p.gpu.tables[0, j].clone()
            p.gpu.tables[0, j] = bad
            o = torch.empty(T, 8, D, dtype=torch.bfloat16, device=DEV)
            m.paged_attn(sh, q, p.gpu, _i32(_packed(news)), _i32(p.lens), o, ws)
            assert m.status_read(ws[:4].view(torch.int32)) == m.MOE_ERR_INVALID_ARG, (bad, j)
            p.gpu.tables[0, j] = old
    # an entry past the context may hold anything
    p.gpu.tables[1, -1] = -2
    assert torch.equal(good, p.attend(q, news, ws=ws))
