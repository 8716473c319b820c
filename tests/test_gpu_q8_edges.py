"""iskv_q8_attention and iskv_q8_append at the edges of what they accept: work
lists past 2^31 steps, blocks of zeros, caps of any size, NaN, short lives of
inputs, waits that run out."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref
from q8_testlib import bound, rows_of, step_floor
from test_gpu_q8_attention import Case

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def test_a_head_with_more_than_two_to_the_31_steps():
    """270000 bf16 queries of 8 heads over as many tokens, announced as single
    ones: a tile of one query, 8438 steps each, 2.28e9 steps of one head.  Rows at
    both ends and in the middle are checked."""
    import online_rank_kv_b200 as ik
    n, heads = 270000, 8
    pages = -(-n // 64)
    gen = torch.Generator(device="cuda").manual_seed(31)
    k = torch.randint(-127, 128, (pages, 1, 64, 128), generator=gen, device="cuda", dtype=torch.int8)
    v = torch.randint(-127, 128, (pages, 1, 64, 128), generator=gen, device="cuda", dtype=torch.int8)
    ks, vs = [2.0 ** torch.randint(-9, -6, (pages, 1), generator=gen, device="cuda").float() for _ in range(2)]
    q = torch.randn(n, heads, 128, generator=gen, device="cuda", dtype=torch.bfloat16)
    out = ik.Q8Pages.of(k, v, ks, vs).attention(q, _i32(np.arange(pages)[None]), _i32([n]), _i32([0, n]), max_new=1)
    kk = (k.float() * ks[..., None, None]).reshape(-1, 1, 128).double().cpu().numpy()
    vv = (v.float() * vs[..., None, None]).reshape(-1, 1, 128).double().cpu().numpy()
    for i in (0, 1, 63, 134999, 254489, n - 1):
        o, mass, size = ref.attention(q[i:i + 1].double().cpu().numpy(), kk[:i + 1], vv[:i + 1], 128 ** -0.5)
        # fp16's smallest steps (step_floor): 2^-39 sum |c| max s, and the largest scale is 4 times the smallest
        floor = 2.0 ** -37 * np.abs(vv[:i + 1]).sum(0)
        assert (np.abs(out[i].double().cpu().numpy() - o[0]) <= (bound(o, mass, size, torch.bfloat16) + floor)[0]).all(), i
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("kv_heads,mod", [(2, {}), (5, dict(cap=20.0)), (2, dict(window=40))])
def test_many_short_prompts_in_a_row(kv_heads, mod):
    """Some ten pieces of one to eleven pages per CTA: step descriptions are handed
    round and round the prompt kernel's ring, first steps close behind last ones."""
    rng = np.random.default_rng(32)
    lens = rng.integers(40, 700, 420).tolist()
    c = Case(lens, [int(rng.integers(33, 41)) for _ in lens], kv_heads, 4, ref.INT8, seed=33)
    c.check(**mod)
    a = c.run(**mod)
    for _ in range(20):
        assert torch.equal(a, c.run(**mod))
    assert c.store().status() == 0


WAITS = r"""
import sys
sys.path[:0] = [sys.argv[1], sys.argv[1] + "/tests"]
import torch
import online_rank_kv_b200 as ik
from test_gpu_q8_attention import Case
from oracle import paged_q8 as ref
for code in (ref.INT8, ref.E4M3):
    for lens, dtype, new, mod in (([3000, 900, 160], "bf16", 1, {}), ([3000, 900, 160], "f32", 6, {}),
                                  ([3000, 900, 160], "f32", 40, dict(cap=20.0)),
                                  ([3000, 900, 160], "bf16", 150, {}),
                                  ([3000, 900, 160], "bf16", 150, dict(window=200, cap=20.0)),
                                  ([60000, 40000, 9000], "bf16", 1, {}), ([60000, 40000, 9000], "f32", 40, dict(cap=20.0)),
                                  ([60000, 40000, 9000], "bf16", 150, {})):
        c = Case(lens, [new] * 3, 2, 4, code, dtype, seed=34)
        for _ in range(2):
            out = c.run(**mod)
            torch.cuda.synchronize()
            print("call", sum(lens), dtype, new, c.store().status(), flush=True)
x = torch.ones(256, 256, device="cuda")
assert ((x @ x) == 256).all()
store = ik.Q8Pages(2, 2)
i32 = dict(dtype=torch.int32, device="cuda")
store.append(torch.ones(3, 2, 128, device="cuda"), torch.ones(3, 2, 128, device="cuda"), torch.arange(3, **i32))
assert store.status() == 0 and (store.k[0, :, :3] == 127).all()
print("alive")
"""


def test_waits_that_run_out_are_reported_and_leave_the_context_usable():
    """A process whose pipeline waits may take one cycle (the waits that let
    copies and products in flight end keep their limit): calls report the
    timeout, none hangs, and the device goes on.  (A step of fp32
    queries takes longer than the copies of the two steps behind it, and short
    requests have few waits: theirs may not run out.)"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, ISKV_TEST_PIPELINE_WAIT_CYCLES="1")
    out = subprocess.run([sys.executable, "-c", WAITS, root], env=env, capture_output=True, text=True, timeout=240)
    assert out.returncode == 0, out.stderr[-2000:]
    lines = out.stdout.split("\n")
    calls = [line.split() for line in lines if line.startswith("call")]
    assert len(calls) == 32 and all(c[-1] in ("0", "-8") for c in calls), out.stdout
    for size, dtype, new, status in [c[1:] for c in calls]:
        assert status == "-8" or dtype == "f32" or int(size) < 10000, out.stdout
    assert "alive" in lines


ZERO_PAGES = [[0], [1], [0, 1], [5], [0, 2, 4, 6, 8, 10, 12, 14], [15], list(range(1, 15)), list(range(16))]


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("zeros", range(len(ZERO_PAGES)))
@pytest.mark.parametrize("spread", [2.0 ** -20, 2.0 ** -40, 2.0 ** 40])
@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("f32", 3), ("bf16", 150)])
def test_pages_without_values_beside_small_ones(code, zeros, spread, dtype, new):
    """Pages of scale 0 count in the denominator and in nothing else: they do not
    take bits from pages whose values are small (or weigh nothing beside large
    ones).  Half of them hold codes: what scale 0 multiplies is zero."""
    c = Case([1000, 300], [new, new], 2, 4, code, dtype, seed=37, spread=spread)
    for b, width in ((0, 16), (1, 5)):
        for j in ZERO_PAGES[zeros]:
            if j < width:
                p = c.table[b, j]
                c.vs[p] = 0
                if j % 2 == 0:
                    c.vc[p] = 0
    c.check()


@pytest.mark.parametrize("lead", [31, 32, 33, 70])
@pytest.mark.parametrize("new", [1, 200])
def test_many_pages_without_values_in_front(lead, new):
    c = Case([80 * 64], [new], 1, 8, ref.INT8, seed=38, spread=2.0 ** -30)
    c.vs[c.table[0, :lead]] = 0
    c.vc[c.table[0, :lead]] = 0
    c.check()


@pytest.mark.parametrize("new", [1, 200])
def test_hidden_pages_do_not_weigh_pages_without_values(new):
    """A sliding window over pages without values and pages 98 powers of two
    apart, which no query sees together."""
    c = Case([900], [new], 2, 4, ref.INT8, seed=39)
    c.vs[:] = np.float32(2.0 ** 60)
    c.vs[c.table[0, ::3]] = np.float32(2.0 ** -38)
    c.vs[c.table[0, 1::3]] = 0
    c.check(window=30)


def _capped(c, cap, d=None):
    """Outputs and bounds of a capped call; d: the scores' error, bound()'s without
    a term for the cap where None."""
    outs, tols, at = [], [], 0
    for b, (n, m) in enumerate(zip(c.lens, c.new)):
        k, v = (rows_of(x, s, c.table[b], n, c.code) for x, s in ((c.kc, c.ks), (c.vc, c.vs)))
        o, mass, size = ref.attention(c.q[at:at + m].double().cpu().numpy(), k, v, 128 ** -0.5, cap)
        if d is None:
            tol = bound(o, mass, size, c.dtype)
        else:
            tol = 2.0 ** -23 * np.abs(o) + (2.0 ** -20 + 3.0 * d(size)) * mass
        outs.append(o)
        tols.append(tol + step_floor(c.vc, c.vs, c.table[b], n, c.code, c.heads, c.dtype))
        at += m
    return np.concatenate(outs), np.concatenate(tols)


@pytest.mark.parametrize("cap", [50.0, 1e3, 1e6, 1e30, 3e38])
@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("bf16", 150), ("f32", 1), ("f32", 40)])
def test_caps_of_any_size(cap, dtype, new):
    """Scores of up to some 10 under caps of up to fp32's largest number, within the
    bound of uncapped ones.  (A cap's own error is at most 2^-20 of the score, as in
    the next test, and the bound's 2^-16 size holds 2^-17 size more than the sums.)"""
    c = Case([400, 130], [min(new, 130)] * 2, 2, 4, ref.INT8, dtype, seed=35, gain=0.6)
    got = c.run(cap=cap).double().cpu().numpy()
    out, tol = _capped(c, cap)
    assert (np.abs(got - out) <= tol).all()


@pytest.mark.parametrize("cap", [0.5, 5.0, 50.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("new", [1, 40])
def test_a_caps_error_goes_by_the_score(cap, new):
    """fp32 queries of one element each, a power of two: scores without rounding
    but for their scale (4 of 2^-24), the cap (2^-20: below half of it a polynomial
    of 2^-22 and its roundings, else 1 - 2 / (1 + e^2t), off by some 4 of 2^-23 where
    the cap is at most twice the score) and two products behind it: 2^-19 of the
    score in all, and 2^-20 for the exponential and the value's scale."""
    c = Case([400, 130], [new] * 2, 2, 4, ref.INT8, "f32", seed=36)
    c.q.zero_()
    at = torch.arange(c.q.shape[0] * c.heads, device="cuda").view(-1, c.heads, 1) * 37 % 128
    c.q.scatter_(2, at, 64.0)          # scores within +-11
    got = c.run(cap=cap).double().cpu().numpy()
    out, tol = _capped(c, cap, d=lambda size: 2.0 ** -19 * size + 2.0 ** -20)
    assert (np.abs(got - out) <= tol).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("f32", 5), ("bf16", 150)])
@pytest.mark.parametrize("mod", [{}, dict(cap=20.0), dict(window=1)])
def test_queries_that_are_not_finite_give_nan_in_their_rows(bad, dtype, new, mod):
    """Wherever the row's keys lie (a first token sees one key only): NaN where the
    formula gives NaN or +infinity for a score that it sees.  Scores that are all
    finite (infinities under a cap are +-cap) give the formula's output, or NaN where
    0 x infinity came into it; the other rows are as ever."""
    c = Case([new, 500, 8 * 64 + 1], [new] * 3, 2, 4, ref.INT8, dtype, seed=40)
    where = [(i, (3 * i) % c.heads) for i in range(0, 3 * new, 1 if new < 10 else 7)]
    clean = c.q.clone()
    for i, h in where:
        c.q[i, h, (5 * i) % 128] = bad
    q = c.q.double().cpu().numpy()
    got = c.run(**mod).double().cpu().numpy()
    c.q = clean
    out, tol = c.want(**mod)
    rows, sure = np.zeros(got.shape[:2], dtype=bool), 0
    for i, h in where:
        rows[i, h] = True
        b, j = divmod(i, new)
        k, v = (rows_of(x, s, c.table[b], c.lens[b], c.code)[:, h // 4] for x, s in ((c.kc, c.ks), (c.vc, c.vs)))
        on = ref.visible(c.lens[b], new, mod.get("window", 0), 0)[j]
        with np.errstate(all="ignore"):
            x = 128 ** -0.5 * (k[on] @ q[i, h])
            if "cap" in mod:
                x = 20.0 * np.tanh(x / 20.0)
        if not (x < np.inf).all():
            sure += 1
            assert np.isnan(got[i, h]).all()
        elif np.isfinite(x).all():
            w = np.exp(x - x.max())
            w /= w.sum()
            o, mass = w @ v[on], w @ np.abs(v[on])
            near = np.abs(got[i, h] - o) <= bound(o, mass, np.full(1, 20.0), c.dtype, 20.0)
            assert near.all() or np.isnan(got[i, h]).all()
    assert sure or bad < 0 or "cap" in mod
    assert (np.abs(got - out) <= tol)[~rows].all()


@pytest.mark.parametrize("dtype,new", [("bf16", 4), ("f32", 4), ("bf16", 150)])
def test_queries_that_are_not_finite_and_see_nothing_give_zeros(dtype, new):
    c = Case([2, 90], [new, new], 2, 4, ref.INT8, dtype, seed=41)
    c.q[0, 1, 2] = float("nan")
    got = c.run()
    assert (got[:new - 2] == 0).all() and torch.isfinite(got).all()


def test_inputs_dropped_after_a_call_on_another_stream():
    """A call on a given stream holds its inputs until that stream has passed it:
    what the current stream allocates next does not get their memory before."""
    import online_rank_kv_b200 as ik
    gen = torch.Generator(device="cuda").manual_seed(43)
    n, kv, heads = 300, 2, 8
    make = lambda h, dt: torch.randn(n, h, 128, generator=gen, device="cuda").to(dt)
    k, v, q = make(kv, torch.float32), make(kv, torch.float32), make(heads, torch.bfloat16)
    table, slots = _i32([[4, 2, 0, 1, 3]]), _i32([64 * [4, 2, 0, 1, 3][t // 64] + t % 64 for t in range(n)])
    lens, cu, prefix, add = _i32([n]), _i32([0, n]), _i32([20]), _i32([n])
    slopes = torch.full((heads,), 0.25, device="cuda")
    free, n_free = _i32([3, 1, 0, 2, 4]), _i32([5])

    def run(stream, copies):
        pages = ik.Q8Pages(5, kv)
        state = torch.full((1, 5), -1, dtype=torch.int32, device="cuda"), free.clone(), n_free.clone()
        out, plan = torch.zeros_like(q), ik.PagePlan.empty(1, n)
        torch.cuda.synchronize()
        if stream is not None:
            with torch.cuda.stream(stream):
                torch.cuda._sleep(40_000_000)          # some 20 ms
        hold = []

        def dropped(*tensors):
            """Fresh copies of a call's inputs; the ones of the call before go."""
            here = [t.clone() for t in tensors]
            if copies:
                torch.cuda.current_stream().synchronize()
            else:
                hold.append(here)
            return here
        ik.page_plan(*dropped(0 * lens, add), *state, out=plan, stream=stream)
        junk = [torch.full_like(t, 9) for t in (lens, add) for _ in range(4)]
        pages.append(*dropped(k, v, slots), stream=stream)
        junk += [torch.full_like(t, 9) for t in (k, v, slots) for _ in range(4)]
        a = dropped(q, table, lens, cu, prefix, slopes)
        pages.attention(*a[:4], max_new=n, prefix=a[4], slopes=a[5], out=out, stream=stream)
        del a
        junk += [torch.full_like(t, 9) for t in (q, table, lens, cu, prefix, slopes) for _ in range(4)]
        torch.cuda.synchronize()
        assert pages.status() == 0 and plan.status.item() == 0
        return pages.k, pages.k_scale, pages.v, out, plan.lens, plan.slots, state[0]
    want = run(None, False)
    got = run(torch.cuda.Stream(), True)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_pages_dropped_after_a_call_on_another_stream():
    import online_rank_kv_b200 as ik
    side, pages = torch.cuda.Stream(), ik.Q8Pages(200, 8)
    x, slots = torch.randn(12800, 8, 128, device="cuda"), _i32(np.arange(12800))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
    pages.append(x, x, slots, stream=side)
    del pages
    junk = [torch.full((200, 8, 64, 128), 9, dtype=torch.int8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert all((j == 9).all() for j in junk)


def test_status_waits_for_calls_on_other_streams():
    import online_rank_kv_b200 as ik
    side, pages = torch.cuda.Stream(), ik.Q8Pages(2, 2)
    x, slots = torch.zeros(3, 2, 128, device="cuda"), _i32([0, 1, 2])
    pages.append(x, x, slots)                  # (the kernel is loaded before the wait begins)
    assert pages.status() == 0
    x.fill_(float("nan"))
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)         # some 100 ms
    pages.append(x, x, slots, stream=side)
    assert pages.status() == -9


@pytest.mark.parametrize("kv_heads", [1, 2])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_row_whatever_its_token_stride(kv_heads, dtype):
    """A single row has no next one: its token stride is whatever a view left."""
    import online_rank_kv_b200 as ik
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    gen = torch.Generator(device="cuda").manual_seed(42)
    k, v = [torch.randn(1, kv_heads, 128, generator=gen, device="cuda").to(dt) for _ in range(2)]
    q = torch.randn(1, 2 * kv_heads, 128, generator=gen, device="cuda").to(dt)
    slots, table, lens, cu = _i32([64]), _i32([[1]]), _i32([1]), _i32([0, 1])

    def odd(x):
        y = torch.as_strided(x, x.shape, (1, 128, 1))
        assert y.stride(0) == 1
        return y
    got = []
    for f in (lambda x: x, odd):
        store = ik.Q8Pages(2, kv_heads)
        store.append(f(k), f(v), slots)
        got.append((store.k.clone(), store.v.clone(), store.attention(f(q), table, lens, cu, max_new=1)))
        assert store.status() == 0
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("new,code", [(1, ref.INT8), (1, ref.E4M3), (40, ref.INT8), (40, ref.E4M3)])
def test_each_call_reads_what_the_one_before_wrote(new, code):
    """Page plan, append and attention with nothing between them, again and again:
    the queries and rows are the attention's last output, the table, lengths and
    slots the plan's, and the pages' scales grow at every step.  The same bits as
    with a synchronize after every call."""
    import online_rank_kv_b200 as ik
    batch, steps, heads = 2, 25, 4
    n = batch * new

    def run(sync):
        pages = ik.Q8Pages(40, heads, code)
        table, free, plan = _i32(np.full((batch, 20), -1)), _i32(np.arange(40)), ik.PagePlan.empty(batch, n)
        plan.lens.zero_()
        plan.n_free.fill_(40)
        add = _i32([new] * batch)
        gen = torch.Generator(device="cuda").manual_seed(44)
        x = [torch.randn(n, heads, 128, generator=gen, device="cuda").bfloat16() for _ in range(2)]
        rows = [torch.randn(n, heads, 128, generator=gen, device="cuda").bfloat16() * 1.3 ** i for i in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            ik.page_plan(plan.lens, add, table, free, plan.n_free, out=plan)
            sync()
            pages.append(rows[i], x[i % 2], plan.slots)
            sync()
            pages.attention(x[i % 2], table, plan.lens, plan.cu, max_new=new, scale=0.05, out=x[(i + 1) % 2])
            sync()
            pages.append(x[(i + 1) % 2], rows[i], plan.slots)      # the same tokens once more
            sync()
        torch.cuda.synchronize()
        assert pages.status() == 0 and plan.status.item() == 0
        return x + [pages.k.view(torch.uint8), pages.v.view(torch.uint8), pages.k_scale, pages.v_scale]
    want = run(torch.cuda.synchronize)
    assert all(torch.isfinite(w).all() for w in want[:2])
    for _ in range(5):
        for a, b in zip(run(lambda: None), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("code", [ref.INT8, ref.E4M3])
@pytest.mark.parametrize("cap", [0.25, 2.0, 8.0])
@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("bf16", 150), ("f32", 9)])
def test_caps_that_bind(code, cap, dtype, new):
    """Scores on both sides of half the cap and far above it."""
    c = Case([400, 1300], [new, new], 2, 4, code, dtype, seed=45, gain=0.6)
    c.q[::3] *= 0.05
    c.q[1::3] *= 4.0
    got = c.run(cap=cap).double().cpu().numpy()
    out, tol = _capped(c, cap)
    assert (np.abs(got - out) <= tol).all()


def test_numbers_beyond_32_bits_are_refused():
    """A window or a largest number of queries that the library's int32 would cut."""
    import online_rank_kv_b200 as ik
    store = ik.Q8Pages(2, 2)
    x = torch.ones(100, 2, 128, device="cuda")
    store.append(x, x, _i32(np.arange(100)))
    q, args = torch.ones(1, 4, 128, device="cuda"), (_i32([[0, 1]]), _i32([100]), _i32([0, 1]))
    for kw in (dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(max_new=2 ** 32 + 1), dict(max_new=2 ** 31),
               dict(window=-2 ** 32)):
        with pytest.raises(ValueError):
            store.attention(q, *args, **dict(dict(max_new=1), **kw))
    a = store.attention(q, *args, max_new=1, window=2 ** 31 - 1)
    assert torch.equal(a, store.attention(q, *args, max_new=1))


@pytest.mark.parametrize("new", [1, 40])
def test_calls_on_given_streams_inside_a_capture(new):
    """A captured step whose calls name their streams, one of them forked off the
    capturing one, with temporary inputs: replayed with other lengths and rows, it
    gives what eager calls give."""
    import online_rank_kv_b200 as ik
    batch, kv, heads = 3, 2, 8
    n = batch * new
    gen = torch.Generator(device="cuda").manual_seed(46)

    class State:
        def __init__(self):
            self.table, self.free = _i32(np.full((batch, 12), -1)), _i32(np.arange(40))
            self.plan = ik.PagePlan.empty(batch, n)
            self.plan.lens.zero_()
            self.plan.n_free.fill_(40)
            self.add = _i32([new] * batch)
            self.pages = ik.Q8Pages(40, kv, ik.CODE_E4M3)
            self.x = torch.zeros(n, heads + 2 * kv, 128, device="cuda", dtype=torch.bfloat16)
            self.out = torch.zeros(n, heads, 128, device="cuda", dtype=torch.bfloat16)

        def step(self, side):
            here = torch.cuda.current_stream()
            ik.page_plan(self.plan.lens, self.add, self.table, self.free, self.plan.n_free, out=self.plan, stream=here)
            k = self.x[:, heads:heads + kv] * 2
            if side is not None:
                side.wait_stream(here)
            self.pages.append(k, self.x[:, heads + kv:], self.plan.slots, stream=side)
            q = self.x[:, :heads] + 0
            if side is not None:
                side.wait_stream(here)
            got = self.pages.attention(q, self.table, self.plan.lens, self.plan.cu, max_new=new, stream=side)
            if side is not None:
                here.wait_stream(side)
            self.out.copy_(got)
    eager, captured, side = State(), State(), torch.cuda.Stream()
    captured.add.zero_()
    captured.step(None)
    captured.add.fill_(new)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured.step(side)
    for i in range(8):
        x = torch.randn(eager.x.shape, generator=gen, device="cuda").bfloat16()
        for s in (eager, captured):
            s.x.copy_(x)
            s.add.copy_(_i32([new, i % 2, 0]))
        eager.step(None)
        graph.replay()
        torch.cuda.synchronize()
        m = int(eager.plan.cu[-1])
        assert torch.equal(eager.plan.lens, captured.plan.lens) and torch.equal(eager.plan.slots, captured.plan.slots)
        assert torch.equal(eager.out[:m], captured.out[:m])
        assert torch.equal(eager.pages.k.view(torch.uint8), captured.pages.k.view(torch.uint8))
    assert captured.pages.status() == 0 and captured.plan.status.item() == 0


@pytest.mark.parametrize("scale", [1e-40, 1e-45, float("nan"), float("inf"), -1.0])
@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("f32", 3), ("bf16", 130)])
def test_hidden_pages_read_no_scale(scale, dtype, new):
    """A table entry outside the pool hides its tokens, whatever stands in the
    scales of pages that nobody holds (page 0 among them)."""
    c = Case([640, 300], [new, new], 2, 4, ref.INT8, dtype, seed=47)
    spare = next(p for p in range(c.kc.shape[0]) if p and p not in c.table)
    for x in (c.kc, c.ks, c.vc, c.vs):
        x[spare] = x[0]
    c.table[c.table == 0] = spare
    want = Case([640, 300], [new, new], 2, 4, ref.INT8, dtype, seed=47).run()
    c.ks[0], c.vs[0] = scale, scale
    assert torch.equal(c.run(), want)
    c.table[0, 3], c.table[1, 1] = -1, 10 ** 6
    got = c.run()
    c.ks[0], c.vs[0], c.store_t = 1.0, 1.0, None
    assert torch.isfinite(got).all() and torch.equal(got, c.run())
