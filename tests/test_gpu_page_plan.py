"""iskv_page_plan against the reference: block tables, the stack of free pages,
slot maps, refusals as a whole, captured and replayed steps."""

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _step_both(lens, add, table, free, n_free, tokens, in_place=False):
    """One step on both sides; compares every output and returns the new state."""
    import online_rank_kv_b200 as ik
    t_ref, f_ref = table.copy(), free.copy()
    want = ref.page_plan(lens, add, t_ref, f_ref, n_free, tokens)
    d_lens, d_table, d_free, d_n = _dev(lens), _dev(table), _dev(free), _dev([n_free])
    out = ik.PagePlan.empty(len(lens), tokens)
    for t in (out.lens, out.cu, out.slots, out.n_free, out.status):
        t.fill_(-77)
    if in_place:
        out.lens, out.n_free = d_lens, d_n
    ik.page_plan(d_lens, _dev(add), d_table, d_free, d_n, out=out)
    torch.cuda.synchronize()
    assert out.status.item() == want[4]
    assert out.lens.tolist() == want[0]
    assert out.cu.tolist() == want[1]
    assert out.slots.tolist() == want[2]
    assert out.n_free.item() == want[3]
    np.testing.assert_array_equal(d_table.cpu().numpy(), t_ref)
    np.testing.assert_array_equal(d_free.cpu().numpy(), f_ref)
    return np.array(want[0]), t_ref, f_ref, want[3], want[4]


@pytest.mark.parametrize("batch,width,pages,seed", [(1, 1, 1, 0), (1, 40, 50, 1), (5, 9, 30, 2), (33, 20, 400, 3),
                                                    (257, 12, 1500, 4), (1025, 5, 3000, 5), (2100, 3, 5000, 6)])
@pytest.mark.parametrize("in_place", [False, True])
def test_many_steps_with_requests_that_come_and_go(batch, width, pages, seed, in_place):
    rng = np.random.default_rng(seed)
    lens = np.zeros(batch, dtype=np.int64)
    table = np.full((batch, width), -1, dtype=np.int32)
    free, n_free = rng.permutation(pages).astype(np.int32), pages
    done = 0
    for step in range(14):
        grow = int(rng.choice([1, 3, 70, 200]))
        add = rng.integers(0, grow + 1, batch)
        add = np.minimum(add, width * 64 - lens)
        add[rng.random(batch) < 0.15] = -1
        # some steps do not fit the pool; both sides refuse them
        tokens = int(np.maximum(add, 0).sum()) + int(rng.integers(0, 4))
        lens, table, free, n_free, status = _step_both(lens, add, table, free, n_free, tokens, in_place)
        done += status == 0
        if status == 0:
            held = [int(table[b, j]) for b in range(batch) for j in range(-(-int(lens[b]) // 64))]
            assert len(set(held)) == len(held) and set(held).isdisjoint(free[:n_free].tolist())
            assert len(held) + n_free == pages
    assert done >= 3


def test_long_prompts_over_several_clusters_of_slots():
    """Slot counts on both sides of every cluster size (1, 2, 4, 8 CTAs)."""
    for tokens in (2047, 2048, 2049, 4097, 8193, 40000):
        width = -(-tokens // 64) + 1
        table = np.full((3, width), -1, dtype=np.int32)
        table[1, :2] = [7, 3]
        free = np.setdiff1d(np.arange(width * 3), [7, 3]).astype(np.int32)
        n = len(free)
        free = np.concatenate([free, [0, 0]]).astype(np.int32)
        add = [tokens // 3, tokens - tokens // 3 - 5, 5]
        *_, status = _step_both([0, 100, 0], add, table, free, n, tokens + 2)
        assert status == 0


@pytest.mark.parametrize("change,code", [
    (dict(lens=[-1, 5]), -1), (dict(lens=[5, 4 * 64 + 1]), -1), (dict(add=[-2, 1]), -1), (dict(n_free=-1), -1),
    (dict(n_free=9), -1), (dict(add=[300, 1]), -2), (dict(add=[100, 150], tokens=249), -2),
    (dict(n_free=2, add=[250, 1]), -2), (dict(lens=[256, 256], add=[-1, -1], n_free=4), -1),
    (dict(add=[2 ** 31 - 1, 2 ** 31 - 1]), -2), (dict(lens=[-1, 5], add=[10 ** 6, 1]), -1)])
def test_refused_steps_change_nothing(change, code):
    a = dict(lens=[0, 70], add=[60, 1], table=np.array([[-1] * 4, [5, 6, -1, -1]], dtype=np.int32),
             free=np.array([0, 1, 2, 3, 4, 7, 0, 0], dtype=np.int32), n_free=6, tokens=300)
    a.update(change)
    *_, status = _step_both(**a)
    assert status == code


def test_page_numbers_outside_the_pool_give_slots_of_minus_one():
    a = dict(lens=[70, 0], add=[3, 70], table=np.array([[5, 900], [-1, -1]], dtype=np.int32),
             free=np.array([4, -3, 1, 0], dtype=np.int32), n_free=3, tokens=80)
    _step_both(**a)


@pytest.mark.parametrize("batch,tokens", [(0, 0), (0, 5), (1, 0), (3, 0)])
def test_empty_batches_and_steps(batch, tokens):
    _step_both([64] * batch, [0] * batch, np.zeros((batch, 2), dtype=np.int32), np.arange(4, dtype=np.int32), 2, tokens)


def test_a_captured_step_replays_with_other_lengths():
    import online_rank_kv_b200 as ik
    batch, width, pages = 6, 8, 48
    lens, add, n_free = _dev([0] * batch), _dev([1] * batch), _dev([pages])
    table, free = _dev(np.full((batch, width), -1)), _dev(np.arange(pages))
    out = ik.PagePlan.empty(batch, 200)
    out.lens, out.n_free = lens, n_free
    ik.page_plan(lens, add, table, free, n_free, out=out)       # warm
    lens.zero_()
    n_free.fill_(pages)
    free.copy_(_dev(np.arange(pages)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ik.page_plan(lens, add, table, free, n_free, out=out)
    r_lens, r_table, r_free, r_n = [0] * batch, np.full((batch, width), -1, dtype=np.int32), np.arange(pages, dtype=np.int32), pages
    table.fill_(-1)
    rng = np.random.default_rng(9)
    for _ in range(8):
        a = rng.integers(-1, 34, batch)
        add.copy_(_dev(a))
        graph.replay()
        torch.cuda.synchronize()
        r_lens, cu, slots, r_n, status = ref.page_plan(r_lens, a, r_table, r_free, r_n, 200)
        assert (out.status.item(), lens.tolist(), out.cu.tolist(), out.slots.tolist(), n_free.item()) == \
            (status, r_lens, cu, slots, r_n)
        np.testing.assert_array_equal(table.cpu().numpy(), r_table)
        np.testing.assert_array_equal(free.cpu().numpy(), r_free)


def test_the_largest_batch():
    rng = np.random.default_rng(40)
    batch, width = 8192, 3
    lens = rng.integers(0, 64 * width + 1, batch)
    add = np.minimum(rng.integers(-1, 9, batch), 64 * width - lens)
    need = int((-(-lens // 64)).sum())
    table = np.full((batch, width), -1, dtype=np.int32)
    order, at = rng.permutation(need + 9000).astype(np.int32), 0
    for b in range(batch):
        k = -(-int(lens[b]) // 64)
        table[b, :k] = order[at:at + k]
        at += k
    free = np.concatenate([order[at:], np.zeros(at, dtype=np.int32)])
    *_, status = _step_both(lens, add, table, free, 9000, int(np.maximum(add, 0).sum()) + 3, in_place=True)
    assert status == 0


@pytest.mark.parametrize("refused", [False, True])
def test_as_many_slots_as_an_int32_counts(refused):
    import online_rank_kv_b200 as ik
    n = 2 ** 31 - 1
    if torch.cuda.mem_get_info()[0] < 4 * n + (2 << 30):
        pytest.skip("needs 8 GiB for the slots")
    out = ik.PagePlan.empty(2, n)
    out.slots.fill_(-77)
    table, free = torch.full((2, 4), -1, dtype=torch.int32, device="cuda"), _dev(np.arange(8))
    ik.page_plan(_dev([0, 0]), _dev([100, 257 if refused else 30]), table, free, _dev([8]), out=out)
    torch.cuda.synchronize()
    assert out.status.item() == (-2 if refused else 0)
    assert out.cu.tolist() == ([0, 0, 0] if refused else [0, 100, 130])
    first = 0 if refused else 130
    want = [] if refused else [7 * 64 + i for i in range(64)] + [6 * 64 + i for i in range(36)] + [5 * 64 + i for i in range(30)]
    assert out.slots[:first].tolist() == want
    assert int(out.slots[first:].max()) == -1 and int(out.slots[first:].min()) == -1
    assert free.tolist() == list(range(8))
