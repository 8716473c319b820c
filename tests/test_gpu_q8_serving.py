"""The paged 8-bit cache as a server uses it: page tables, writes and attention
of the same requests step after step, eagerly and as one captured graph."""

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref
from q8_testlib import bound, np_codes, rows_of

pytestmark = pytest.mark.gpu
HEADS, KV, PAGES, WIDTH = 8, 2, 40, 8


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Server:
    """A batch of requests on the GPU beside the reference's state."""

    def __init__(self, batch, code, tokens):
        import online_rank_kv_b200 as ik
        self.ik, self.code, self.batch, self.tokens = ik, code, batch, tokens
        self.lens, self.add, self.n_free = _i32([0] * batch), _i32([0] * batch), _i32([PAGES])
        self.table, self.free = _i32(np.full((batch, WIDTH), -1)), _i32(np.arange(PAGES))
        self.plan = ik.PagePlan.empty(batch, tokens)
        self.plan.lens, self.plan.n_free = self.lens, self.n_free
        self.layers = [ik.Q8Pages(PAGES, KV, code) for _ in range(2)]
        self.qkv = torch.zeros(tokens, HEADS + 2 * KV, 128, dtype=torch.bfloat16, device="cuda")
        self.outs = [torch.zeros(tokens, HEADS, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.r_lens, self.r_table = [0] * batch, np.full((batch, WIDTH), -1, dtype=np.int32)
        self.r_free, self.r_n = np.arange(PAGES, dtype=np.int32), PAGES
        dt = np.int8 if code == ref.INT8 else np.uint8
        self.r_layers = [[np.zeros((PAGES, KV, 64, 128), dtype=dt), np.zeros((PAGES, KV), dtype=np.float32),
                          np.zeros((PAGES, KV, 64, 128), dtype=dt), np.zeros((PAGES, KV), dtype=np.float32)]
                         for _ in range(2)]

    def step(self):
        """What is enqueued every step (and captured once)."""
        self.ik.page_plan(self.lens, self.add, self.table, self.free, self.n_free, out=self.plan)
        q, k, v = self.qkv[:, :HEADS], self.qkv[:, HEADS:HEADS + KV], self.qkv[:, HEADS + KV:]
        for i, layer in enumerate(self.layers):
            layer.append(k, v, self.plan.slots)
            layer.attention(q, self.table, self.lens, self.plan.cu, max_new=self.tokens, out=self.outs[i])

    def check(self, add):
        torch.cuda.synchronize()
        before = [o for o in self.outs]
        self.r_lens, cu, slots, self.r_n, status = ref.page_plan(self.r_lens, add, self.r_table, self.r_free, self.r_n,
                                                                 self.tokens)
        assert self.plan.status.item() == status == 0
        assert self.lens.tolist() == self.r_lens and self.plan.slots.tolist() == slots
        x = self.qkv.float().cpu().numpy()
        for i, (layer, r) in enumerate(zip(self.layers, self.r_layers)):
            assert ref.append(r[0], r[1], x[:, HEADS:HEADS + KV], slots, self.code) == 0
            assert ref.append(r[2], r[3], x[:, HEADS + KV:], slots, self.code) == 0
            np.testing.assert_array_equal(np_codes(layer.k, self.code), r[0])
            np.testing.assert_array_equal(np_codes(layer.v, self.code), r[2])
            got = before[i].double().cpu().numpy()
            for b in range(self.batch):
                n, m = self.r_lens[b], cu[b + 1] - cu[b]
                if m == 0:
                    continue
                o, mass, size = ref.attention(x[cu[b]:cu[b + 1], :HEADS].astype(np.float64),
                                              rows_of(r[0], r[1], self.r_table[b], n, self.code),
                                              rows_of(r[2], r[3], self.r_table[b], n, self.code), 128 ** -0.5)
                assert (np.abs(got[cu[b]:cu[b + 1]] - o) <= bound(o, mass, size, torch.bfloat16)).all(), (i, b)
            assert layer.status() == 0


def _adds(rng, lens, tokens, batch):
    add = rng.integers(0, tokens // batch + 1, batch)
    add = np.minimum(add, WIDTH * 64 - np.array(lens))
    add[(rng.random(batch) < 0.2) & (np.array(lens) > 200)] = -1
    return add


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("tokens", [5, 400])
@pytest.mark.parametrize("captured", [False, True])
def test_steps_of_a_running_batch(code, tokens, captured):
    rng = np.random.default_rng(tokens + captured)
    s = Server(5, code, tokens)
    g = torch.Generator(device="cuda").manual_seed(1)
    graph = None
    if captured:
        s.step()                       # an empty step: nothing added
        s.check([0] * 5)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
    for _ in range(12):
        add = _adds(rng, s.r_lens, tokens, 5)
        s.add.copy_(_i32(add))
        s.qkv.copy_(torch.randn(s.qkv.shape, generator=g, device="cuda"))
        if graph is not None:
            graph.replay()
        else:
            s.step()
        s.check(add)


def test_two_graphs_of_two_batches_replayed_at_once():
    """Two captured steps with workspaces of their own, on two streams."""
    servers = [Server(5, ref.INT8, 40) for _ in range(2)]
    graphs, g = [], torch.Generator(device="cuda").manual_seed(2)
    for s in servers:
        s.step()
        s.check([0] * 5)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.step()
        graphs.append(graph)
    rng = np.random.default_rng(5)
    streams = [torch.cuda.Stream() for _ in servers]
    for _ in range(6):
        adds = [_adds(rng, s.r_lens, 40, 5) for s in servers]
        for s, a in zip(servers, adds):
            s.add.copy_(_i32(a))
            s.qkv.copy_(torch.randn(s.qkv.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        for s, a in zip(servers, adds):
            s.check(a)


def test_a_chunked_prompt_equals_its_tokens_one_by_one():
    """A prompt in chunks of odd sizes and the same prompt token by token: e4m3
    pages with unchanging scales hold the same codes, and the attention of the
    last token is the same within its bound."""
    import online_rank_kv_b200 as ik
    n = 150
    x = torch.randn(n, HEADS + 2 * KV, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    x[0::64, HEADS:, 0] = 5.0           # each page's largest value in its first row
    x = x.clamp(-5, 5).bfloat16()
    q, k, v = x[:, :HEADS], x[:, HEADS:HEADS + KV], x[:, HEADS + KV:]
    outs, stores = [], []
    for chunks in ([17, 64, 3, 66], [1] * n):
        store = ik.Q8Pages(4, KV, ik.CODE_E4M3)
        lens, table, free, n_free = _i32([0]), _i32([[-1] * 4]), _i32([3, 1, 0, 2]), _i32([4])
        at = 0
        for c in chunks:
            p = ik.page_plan(lens, _i32([c]), table, free, n_free, tokens=c)
            store.append(k[at:at + c], v[at:at + c], p.slots)
            out = store.attention(q[at:at + c], table, p.lens, p.cu, max_new=c)
            lens, n_free, at = p.lens, p.n_free, at + c
        outs.append(out[-1])
        stores.append(store)
    assert torch.equal(stores[0].k.view(torch.int8), stores[1].k.view(torch.int8))
    assert torch.equal(stores[0].v.view(torch.int8), stores[1].v.view(torch.int8))
    s = stores[0]
    table = np.array([2, 0, 1])         # the stack from its top
    kk = rows_of(np_codes(s.k, 1), s.k_scale.cpu().numpy(), table, n, 1)
    vv = rows_of(np_codes(s.v, 1), s.v_scale.cpu().numpy(), table, n, 1)
    o, mass, size = ref.attention(q[-1:].double().cpu().numpy(), kk, vv, 128 ** -0.5)
    for out in outs:
        assert (np.abs(out.double().cpu().numpy() - o[0]) <= bound(o, mass, size, torch.bfloat16)[0]).all()


def test_other_gpus_tensors_are_refused_by_the_binding():
    import online_rank_kv_b200 as ik
    store = ik.Q8Pages(2, KV, ik.CODE_INT8)
    x = torch.zeros(1, KV, 128)
    with pytest.raises(ValueError):
        store.append(x, x, _i32([0]))
    y = x.cuda()
    with pytest.raises(ValueError):
        store.append(y, y, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        store.append(y.half(), y.half(), _i32([0]))
    with pytest.raises(ValueError):
        store.append(y[:, :1], y[:, :1], _i32([0]))
    q = torch.zeros(1, HEADS, 128, device="cuda", requires_grad=True)
    with pytest.raises(ValueError):
        store.attention(q, _i32([[0]]), _i32([1]), _i32([0, 1]), max_new=1)
    with pytest.raises(ik.IskvError):
        store.attention(q.detach(), _i32([[0]]), _i32([1]), _i32([0, 1]), max_new=1, cap=-1.0)
    with pytest.raises(ik.IskvError):
        store.attention(torch.zeros(1, 9 * KV, 128, device="cuda"), _i32([[0]]), _i32([1]), _i32([0, 1]), max_new=1)
    with pytest.raises(ValueError):
        store.attention(q.detach(), _i32([[0]]), _i32([1, 2]), _i32([0, 1]), max_new=1)


def test_calls_follow_one_another_without_a_gap():
    """Many short calls in a row, each reading what the one before wrote, with
    copies and a second stream between them, captured and replayed: the same
    bits as with a synchronize after each call."""
    import online_rank_kv_b200 as ik
    batch, steps = 3, 12
    gen = torch.Generator(device="cuda").manual_seed(7)
    qkv = torch.randn(steps, batch, HEADS + 2 * KV, 128, generator=gen, device="cuda").bfloat16()

    def run(layer, plan, state, outs, sync, side):
        table, free = state
        plan.lens.zero_()
        plan.n_free.fill_(PAGES)
        free.copy_(torch.arange(PAGES, dtype=torch.int32, device="cuda"))
        add = torch.ones(batch, dtype=torch.int32, device="cuda")
        x = torch.empty_like(qkv[0])
        for i in range(steps):
            x.copy_(qkv[i])
            q, k, v = x[:, :HEADS], x[:, HEADS:HEADS + KV], x[:, HEADS + KV:]
            ik.page_plan(plan.lens, add, table, free, plan.n_free, out=plan)
            sync()
            layer.append(k, v, plan.slots)
            sync()
            if side is not None and i % 3 == 1:
                here = torch.cuda.current_stream()
                side.wait_stream(here)
                with torch.cuda.stream(side):
                    layer.attention(q, table, plan.lens, plan.cu, max_new=1, out=outs[i])
                here.wait_stream(side)
            else:
                layer.attention(q, table, plan.lens, plan.cu, max_new=1, out=outs[i])
            sync()
            # what the attention answered is part of the next step's input
            if i + 1 < steps:
                qkv_next = outs[i][:, :KV] * 0.25
                layer.append(qkv_next, qkv_next, plan.slots)
                sync()

    def fresh():
        plan = ik.PagePlan.empty(batch, batch)
        state = (_i32(np.full((batch, WIDTH), -1)), _i32(np.arange(PAGES)))
        outs = [torch.zeros(batch, HEADS, 128, dtype=torch.bfloat16, device="cuda") for _ in range(steps)]
        return ik.Q8Pages(PAGES, KV, ik.CODE_E4M3), plan, state, outs

    want = fresh()
    run(*want, torch.cuda.synchronize, None)
    side = torch.cuda.Stream()
    eager = fresh()
    run(*eager, lambda: None, side)
    torch.cuda.synchronize()
    captured = fresh()
    run(*captured, torch.cuda.synchronize, side)      # buffers in place
    captured[0].k.zero_()
    captured[0].v.zero_()
    captured[0].k_scale.zero_()
    captured[0].v_scale.zero_()
    captured[2][0].fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*captured, lambda: None, side)
    for o in captured[3]:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for got in (eager, captured):
        for a, b in zip(got[3], want[3]):
            assert torch.equal(a, b)
        assert torch.equal(got[0].k.view(torch.uint8), want[0].k.view(torch.uint8))
        assert torch.equal(got[0].v_scale, want[0].v_scale)
        assert got[0].status() == 0
