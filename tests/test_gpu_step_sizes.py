"""Dropout, router and embedding where their launches of large calls begin: sizes
taken from the launch rules (constants of the sources and the GPU's SMs), whole
outputs against the 64-bit forms."""
import numpy as np
import pytest
import torch

import cast_transpose_gb300 as ct
import ops_reference as base
import step_reference as ref
from gpu_util import Guarded, scalar
from test_gpu_embedding import backward as embedding_backward
from test_gpu_embedding import ids
from test_gpu_layer_norm import SEED, SITE, STEP, data, state
from test_gpu_router import Case

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ---- dropout
def check_dropout(rows, cols, dtype, p=0.3, shift=0):
    x = data((rows, cols), dtype, rows + cols)
    want = ref.dropped(x, ref.drop_factor(rows, cols, p, SEED, STEP, SITE))
    g = Guarded(rows * cols, dtype=dtype, offset=shift)
    ct.dropout(x.cuda(), g.t.view(rows, cols), p, state(), SITE)
    torch.cuda.synchronize()
    g.check()
    base.close(g.t.view(rows, cols), want, base.rounded(want, ref.F * want.abs(), dtype), "out")
    y = x.cuda()
    ct.dropout(y, y, p, state(), SITE)
    assert torch.equal(y, g.t.view(rows, cols))


@pytest.mark.parametrize("dtype", [BF, HF, F32])
@pytest.mark.parametrize("cols", [8, 72, 1024, 4104, 8200])
def test_dropout_of_many_whole_groups(cols, dtype):
    """Four groups a thread, twice: from 2048 groups for each SM on."""
    check_dropout(sms() * 2048 * 8 // cols + 5, cols, dtype)


def test_dropout_around_the_first_of_them():
    groups = sms() * 2048
    for n in (groups - 1, groups, groups + 1, groups + 2048 * 3 + 77):
        check_dropout(n, 8, BF)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [257, 4099, 65541])
def test_dropout_of_many_other_rows(cols, dtype):
    """One array of vectors, sixteen steps a warp: from 32768 vectors for each SM on;
    eight below."""
    vectors = sms() * 8 * 256 * 16
    check_dropout(vectors * 8 // cols + 2, cols, dtype)
    if dtype is BF:
        check_dropout(vectors * 8 // cols // 9, cols, dtype)


@pytest.mark.parametrize("rows,cols,shift", [(30011, 100, 0), (20011, 255, 3), (5003, 2056, 1), (3001, 4099, 5)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_dropout_of_any_rows_with_several_to_a_thread(rows, cols, shift, dtype):
    check_dropout(rows, cols, dtype, shift=shift)


def kept(rows, cols, p, site):
    """Which elements of these rows are."""
    group, row = np.meshgrid(np.arange(-(-cols // 8)), np.asarray(rows))
    words = ref.philox((group, row, np.full_like(row, site), np.full_like(row, STEP % 2 ** 32)),
                       (SEED % 2 ** 32, SEED >> 32))
    bits = np.stack([h for w in words for h in (w % 65536, w // 65536)], 2).reshape(len(rows), -1)[:, :cols]
    return bits >= ref.cut_of(p)


@pytest.mark.parametrize("elements,cols", [(2 ** 32, 4095), (2 ** 35, 4096)])
def test_dropout_past_32_bits(elements, cols):
    """More elements, or more groups of eight, than 32 bits count: rows at both ends
    and around each power of two."""
    rows = elements // cols + 3
    x = torch.ones(rows, cols, dtype=BF, device="cuda")
    ct.dropout(x, x, 0.25, state(), 2)
    at = {0, 1, rows - 2, rows - 1}
    for bits in (31, 32, 34, 35):
        at |= {r for r in range(2 ** bits // cols - 1, 2 ** bits // cols + 2) if r < rows}
    at = sorted(at)
    got = x[torch.tensor(at, device="cuda")].cpu()
    del x
    torch.cuda.empty_cache()
    assert np.array_equal((got > 0).numpy(), kept(at, cols, 0.25, 2))
    assert set(got.unique().tolist()) == {0.0, torch.tensor(65536 / (65536 - ref.cut_of(0.25))).to(BF).item()}


# ---- router
MANY = [(9000, 64, 4, F32), (9000, 8, 2, BF), (9000, 33, 3, HF), (5000, 100, 6, F32), (5000, 256, 8, F32),
        (5000, 256, 8, BF), (4000, 512, 40, F32), (3000, 1000, 5, HF)]


@pytest.mark.parametrize("T,E,K,dtype", MANY)
@pytest.mark.parametrize("normalize", [False, True])
def test_router_with_several_tokens_a_warp(T, E, K, dtype, normalize):
    """Forward and backward, padding tokens among them."""
    blocks = sms() * {8: 6, 33: 6, 64: 6, 100: 4, 256: 3, 512: 2, 1000: 1}[E]
    assert T > 8 * blocks
    c = Case(T, E, K, dtype=dtype, normalize=normalize, masked=True)
    c.check()
    c.backward()


@pytest.mark.parametrize("T,E,K", [(9000, 64, 4), (5000, 256, 8), (3000, 1000, 33)])
@pytest.mark.parametrize("normalize", [False, True])
def test_an_expert_twice_in_some_tokens(T, E, K, normalize):
    """What such a token leaves behind is not the next one's."""
    c = Case(T, E, K, normalize=normalize, masked=True)
    w = c.reference()
    for rows in (slice(0, None, 3), slice(T - T // 3, None, 2)):
        w.idx[rows, 1] = w.idx[rows, 0]
    at = w.idx.long().clamp(min=0)
    w.weights = torch.where(w.idx >= 0, w.p.gather(1, at), 0.0)
    if normalize:
        w.weights = torch.where(w.idx >= 0, w.weights / w.weights.sum(1, keepdim=True), 0.0)
    value, err = w.backward(c.dweights, c.dloss)
    dl = torch.empty(T, E, device="cuda")
    ct.moe_router_backward(c.dweights.cuda(), scalar(c.dloss), c.logits.cuda(), w.idx.cuda(), w.counts.cuda(), dl,
                           mask=c.mask.cuda(), **c.kw)
    base.close(dl, value, base.rounded(value, err, F32), "dlogits")


# ---- embedding
@pytest.mark.parametrize("kind", ["text", "uniform", "two", "descending"])
@pytest.mark.parametrize("V,H", [(5000, 72), (70000, 13)])
def test_gradient_of_more_tokens_than_one_cluster_sorts(V, H, kind):
    T = 131072 + 1001
    idx, dout = ids(T, V, kind=kind), data((T, H), BF, 1)
    embedding_backward(idx, dout, V, F32)
    embedding_backward(idx, dout, V, BF, old=data((V, H), BF, 3))


@pytest.mark.parametrize("T", [131072, 131073])
def test_gradient_around_that_number(T):
    idx, dout = ids(T, 3000, dtype=torch.int32), data((T, 24), HF, 1)
    embedding_backward(idx, dout, 3000, F32)
    embedding_backward(idx, dout, 3000, HF, old=data((3000, 24), HF, 3))
