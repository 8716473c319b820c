"""iskv_q8_append against the reference, code for code: fresh and continued
pages, growth of a page's scale, strides, skipped and bad slots, values that
are not finite, zeros, extremes."""

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref
from q8_testlib import np_codes, random_store, to_store

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _check(code, dtype, pages, heads, k, v, slots, store=None, seed=0):
    """k, v torch tensors [n, heads, 128] on the GPU (any token stride)."""
    import online_rank_kv_b200 as ik
    rng = np.random.default_rng(seed)
    c, s = store or (random_store(rng, pages, heads, code), random_store(rng, pages, heads, code))
    kc, ks = (x.copy() for x in c)
    vc, vs = (x.copy() for x in s)
    dk, dv = to_store(kc, code), to_store(vc, code)
    dks, dvs = torch.from_numpy(ks.copy()).cuda(), torch.from_numpy(vs.copy()).cuda()
    pages_ = ik.Q8Pages.of(dk, dv, dks, dvs)
    pages_.append(k, v, torch.tensor(slots, dtype=torch.int32, device="cuda"))
    status = pages_.status()
    w1 = ref.append(kc, ks, k.float().cpu().numpy(), slots, code)
    w2 = ref.append(vc, vs, v.float().cpu().numpy(), slots, code)
    assert status == min(w1, w2)
    np.testing.assert_array_equal(dks.cpu().numpy(), ks)
    np.testing.assert_array_equal(dvs.cpu().numpy(), vs)
    np.testing.assert_array_equal(np_codes(dk, code), kc)
    np.testing.assert_array_equal(np_codes(dv, code), vc)
    return pages_, (kc, ks), (vc, vs)


def _rows(n, heads, dtype, seed, gain=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(2, n, heads, 128, generator=g, device="cuda") * gain
    x[0, ..., 3::32] *= 10
    return x.to(DT[dtype])


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("heads", [1, 3, 8])
@pytest.mark.parametrize("first,n", [(0, 1), (0, 63), (0, 64), (0, 65), (0, 200), (1, 1), (1, 62), (1, 63), (1, 64),
                                     (37, 5), (37, 300), (63, 1), (63, 2), (63, 130)])
def test_one_request_from_any_row_on(code, dtype, heads, first, n):
    pages = 8
    order = np.random.default_rng(n).permutation(pages)
    slots = [int(order[t // 64]) * 64 + t % 64 for t in range(first, first + n)]
    x = _rows(n, heads, dtype, seed=first + n)
    _check(code, dtype, pages, heads, x[0], x[1], slots)


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("n_requests", [1, 7, 90, 700])
def test_one_token_of_many_requests(code, n_requests):
    rng = np.random.default_rng(n_requests)
    order = rng.permutation(n_requests + 2)
    slots = [int(order[b]) * 64 + int(rng.integers(0, 64)) for b in range(n_requests)]
    x = _rows(n_requests, 2, "bf16", seed=n_requests)
    _check(code, "bf16", n_requests + 2, 2, x[0], x[1], slots)


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
def test_ragged_runs_whose_pages_lie_side_by_side(code):
    """Runs that follow each other in the call and in the pool: the next page's
    first row, and a later row of the next page, both begin a run."""
    slots = list(range(60, 64)) + list(range(64, 70)) + list(range(128 + 5, 128 + 9)) + list(range(192, 300)) + [64 * 6 + 63]
    x = _rows(len(slots), 2, "f32", seed=3)
    _check(code, "f32", 8, 2, x[0], x[1], slots)


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
def test_a_page_filled_token_by_token_with_growing_rows(code):
    """Its scale grows many times; every earlier row is coded again each time."""
    import online_rank_kv_b200 as ik
    pages = ik.Q8Pages(3, 2, code)
    kc, ks = np_codes(pages.k, code), pages.k_scale.cpu().numpy()
    vc, vs = np_codes(pages.v, code), pages.v_scale.cpu().numpy()
    for t in range(64):
        x = _rows(1, 2, "bf16", seed=t, gain=1.13 ** t)
        pages.append(x[0], x[1], torch.tensor([64 + t], dtype=torch.int32, device="cuda"))
        ref.append(kc, ks, x[0].float().cpu().numpy(), [64 + t], code)
        ref.append(vc, vs, x[1].float().cpu().numpy(), [64 + t], code)
    assert pages.status() == 0
    np.testing.assert_array_equal(np_codes(pages.k, code), kc)
    np.testing.assert_array_equal(np_codes(pages.v, code), vc)
    np.testing.assert_array_equal(pages.k_scale.cpu().numpy(), ks)
    np.testing.assert_array_equal(pages.v_scale.cpu().numpy(), vs)


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_of_a_fused_projection(code, dtype):
    x = torch.randn(150, 4 + 2 * 3, 128, device="cuda").to(DT[dtype])
    slots = list(range(10, 64)) + list(range(128, 128 + 64)) + list(range(256, 256 + 32))
    _check(code, dtype, 6, 3, x[:, 4:7], x[:, 7:], slots)


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
def test_skipped_and_bad_slots(code):
    x = _rows(9, 2, "f32", seed=5)
    _, _, _ = _check(code, "f32", 3, 2, x[0], x[1], [-1, 10, 11, -1, 64, 192, -2, 2 ** 31 - 1, 129])
    x = _rows(3, 2, "f32", seed=6)
    pages, _, _ = _check(code, "f32", 3, 2, x[0], x[1], [-1, -1, -1])
    assert pages.status() == 0


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_values_that_are_not_finite_are_zeros_and_reported(code, dtype):
    x = _rows(40, 2, dtype, seed=7)
    x[0, 3, 1, 17] = float("inf")
    x[0, 4, 1, 5] = float("nan")
    x[1, 39, 0, 0] = -float("inf")
    x[1, 0] = float("nan")
    pages, (kc, _), _ = _check(code, dtype, 3, 2, x[0], x[1], list(range(70, 110)))
    assert pages.status() == ref.RANGE
    assert kc[1, 1, 9, 17] == 0


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
def test_zeros_extremes_and_ties(code):
    x = torch.zeros(2, 64 * 6, 1, 128, device="cuda")
    x[0, 64:128] = torch.finfo(torch.float32).max
    x[1, 64:128, 0, ::2] = -torch.finfo(torch.float32).max
    x[0, 128:192] = 2.0 ** -64                       # the smallest block that is coded
    x[1, 128:192] = 2.0 ** -65                       # counts as zeros
    x[0, 192:256, 0] = torch.arange(128, device="cuda").float() - 0.5      # halves: ties
    x[0, 192, 0, 0] = 127.0
    x[1, 192:256, 0] = torch.arange(128, device="cuda").float() * 3.5
    x[1, 192, 0, 0] = 448.0
    x[0, 256:320, 0, 1] = 1e-42                      # subnormal beside ordinary values
    x[0, 256:320, 0, 0] = 1.0
    x[1, 256:320, 0, 0] = 448.0 * 2 ** 5 * (1 + 2 ** -20)      # just over a power's reach
    x[1, 320:, 0, 0] = -0.0
    _check(code, "f32", 7, 1, x[0], x[1], list(range(64 * 6)))


def test_the_same_call_twice_changes_nothing_more():
    import online_rank_kv_b200 as ik
    for code in (ref.INT8, ref.E4M3):
        x = _rows(30, 2, "bf16", seed=11, gain=4.0)
        pages, _, _ = _check(code, "bf16", 4, 2, x[0], x[1], list(range(20, 50)))
        before = [t.clone() for t in (pages.k.view(torch.int8), pages.v.view(torch.int8), pages.k_scale, pages.v_scale)]
        pages.append(x[0], x[1], torch.arange(20, 50, dtype=torch.int32, device="cuda"))
        for a, b in zip(before, (pages.k.view(torch.int8), pages.v.view(torch.int8), pages.k_scale, pages.v_scale)):
            assert torch.equal(a, b)
    assert ik.PAGE == 64


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_thousands_of_tokens_in_runs_of_every_length(code, dtype):
    """Enough tokens that a CTA looks after up to 64 of them: runs that start and
    end anywhere in its window, cross into the next one, skipped slots between."""
    rng = np.random.default_rng(31)
    slots, page = [], 0
    while len(slots) < 9000:
        first = int(rng.integers(0, 64))
        n = int(rng.choice([1, 1, 2, 7, 64 - first, 64]))
        slots += [page * 64 + r for r in range(first, min(64, first + n))]
        slots += [-1] * int(rng.integers(0, 3))
        page += 1
    x = _rows(len(slots), 2, dtype, seed=32)
    _check(code, dtype, page + 1, 2, x[0], x[1], slots)


def test_quotients_next_to_a_half():
    """Rows whose quotients by the scale lie within a few ulps of k + 1/2, where a
    product with the reciprocal rounds to the other side."""
    top = np.float32(97.31)
    s = np.float32(top * (np.float32(1) / np.float32(127)))
    k = np.arange(-126, 126).astype(np.float32) + np.float32(0.5)
    rows = np.zeros((64, 1, 128), dtype=np.float32)
    vals = []
    for d in range(-8, 9):
        v = (k * s).astype(np.float32)
        for _ in range(abs(d)):
            v = np.nextafter(v, np.float32(np.inf if d > 0 else -np.inf)).astype(np.float32)
        vals.append(v)
    flat = np.concatenate(vals)[:64 * 128 - 1]
    rows.reshape(-1)[1:1 + flat.size] = flat
    rows[0, 0, 0] = top
    x = torch.from_numpy(rows).cuda()
    _check(ref.INT8, "f32", 2, 1, x, -x, list(range(64)))


def test_a_stream_of_its_own():
    import online_rank_kv_b200 as ik
    x = _rows(70, 2, "bf16", seed=33)
    a, b = ik.Q8Pages(3, 2), ik.Q8Pages(3, 2)
    slots = torch.arange(70, dtype=torch.int32, device="cuda")
    a.append(x[0], x[1], slots)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    b.append(x[0], x[1], slots, stream=s)
    s.synchronize()
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.k_scale, b.k_scale)


def test_one_head_of_a_transposed_tensor():
    """The stride of a dimension of one element says nothing."""
    import online_rank_kv_b200 as ik
    x = torch.randn(1, 70, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    x = x.transpose(0, 1)                       # [70, 1, 128], stride of the head: 70 * 128
    assert x.stride() == (128, 70 * 128, 1)
    slots = torch.arange(70, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    got = []
    for t in (x, x.contiguous().view(70, 128).unsqueeze(1)):
        pages = ik.Q8Pages(2, 1, ik.CODE_INT8)
        pages.append(t, t, slots)
        out = pages.attention(t, torch.tensor([[0, 1]], **i32), torch.tensor([70], **i32), torch.tensor([0, 70], **i32),
                              max_new=70)
        got.append((pages.k, pages.v_scale, out))
    for a, b in zip(*got):
        assert torch.equal(a, b)
