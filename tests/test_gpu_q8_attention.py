"""iskv_q8_attention against float64: single tokens, drafts and prompts over
ragged requests; masks, caps, distance biases, odd sizes, strides, bad pages,
inconsistent lengths, streams and captured graphs."""

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref
from q8_testlib import bound, random_store, rows_of, scattered_table, step_floor, to_store

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


class Case:
    def __init__(self, lens, new, kv_heads, g, code, dtype="bf16", seed=0, extra_pages=3, extra_width=0, gain=0.06,
                 fused=False, spread=1.0, pad=0):
        rng = np.random.default_rng(seed)
        self.lens, self.new, self.code, self.dtype = list(lens), list(new), code, DT[dtype]
        self.kv_heads, self.g, self.heads = kv_heads, g, kv_heads * g
        pages = sum(-(-n // 64) for n in lens) + extra_pages
        width = max([1] + [-(-n // 64) for n in lens]) + extra_width
        self.kc, self.ks = random_store(rng, pages, kv_heads, code)
        self.vc, self.vs = random_store(rng, pages, kv_heads, code, spread)
        self.table = scattered_table(rng, lens, width, pages)
        n = sum(new) + pad
        q = torch.from_numpy(rng.standard_normal((max(n, 1), self.heads + 2, 128)) * gain * 8)
        q = q.to(self.dtype).cuda()
        self.q = q[:, 1:1 + self.heads][:n] if fused else q[:, 1:1 + self.heads][:n].contiguous()
        self.store_t = None

    def store(self):
        import online_rank_kv_b200 as ik
        if self.store_t is None:
            self.store_t = ik.Q8Pages.of(to_store(self.kc, self.code), to_store(self.vc, self.code),
                                         torch.from_numpy(self.ks.copy()).cuda(), torch.from_numpy(self.vs.copy()).cuda())
        return self.store_t

    def run(self, max_new=None, prefix=None, slopes=None, lens=None, **kw):
        def i32(x):
            return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
        cu = np.concatenate([[0], np.cumsum(self.new)])
        return self.store().attention(
            self.q, i32(self.table).reshape(len(self.lens), -1), i32(self.lens if lens is None else lens), i32(cu),
            max_new=max_new or max(self.new + [1]), prefix=None if prefix is None else i32(prefix),
            slopes=None if slopes is None else torch.tensor(slopes, dtype=torch.float32, device="cuda"), **kw)

    def want(self, cap=0.0, slopes=None, window=0, prefix=None, scale=128 ** -0.5):
        outs, bounds, at = [], [], 0
        for b, (n, m) in enumerate(zip(self.lens, self.new)):
            q = self.q[at:at + m].double().cpu().numpy()
            k = rows_of(self.kc, self.ks, self.table[b], n, self.code)
            v = rows_of(self.vc, self.vs, self.table[b], n, self.code)
            o, mass, size = ref.attention(q, k, v, scale, cap, slopes, window, 0 if prefix is None else prefix[b])
            bias = 0.0 if slopes is None else 64.0      # beyond it a weight is nothing
            outs.append(o)
            floor = step_floor(self.vc, self.vs, self.table[b], n, self.code, self.heads, self.dtype) if n else 0.0
            bounds.append(bound(o, mass, size, self.dtype, cap, bias) + floor)
            at += m
        return np.concatenate(outs), np.concatenate(bounds)

    def check(self, max_new=None, **kw):
        got = self.run(max_new=max_new, **kw)
        assert got.dtype == self.dtype and got.shape == self.q.shape
        got = got.double().cpu().numpy()[:sum(self.new)]
        out, tol = self.want(**kw)
        worst = (np.abs(got - out) / tol).max() if out.size else 0.0
        assert np.isfinite(got).all()
        assert worst <= 1.0, worst
        return worst


CODES = [ref.INT8, ref.E4M3]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [1, 2, 3, 4, 7, 8])
def test_single_tokens_of_ragged_requests(code, dtype, g):
    lens = [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 500, 1000, 2049]
    Case(lens, [1] * len(lens), 2, g, code, dtype, seed=g).check()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("length", [1, 33, 64, 1000, 5000, 20000])
def test_one_token_of_one_request(code, length):
    Case([length], [1], 8, 4, code, seed=length).check()


@pytest.mark.parametrize("kv_heads,length", [(1, 30000), (1, 100), (5, 3001)])
def test_one_request_shared_by_the_whole_gpu(kv_heads, length):
    Case([length], [1], kv_heads, 8, ref.INT8, "f32", seed=length).check()


@pytest.mark.parametrize("code", CODES)
def test_many_short_requests_per_warp(code):
    rng = np.random.default_rng(1)
    lens = rng.integers(1, 70, 1300).tolist()
    Case(lens, [1] * len(lens), 3, 4, code, seed=2).check()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [1, 3, 4, 8])
def test_drafts_of_several_tokens(code, dtype, g):
    lens, new = [5, 9, 64, 300, 1111, 40, 77], [5, 2, 1, 8, 7, 0, 3]
    Case(lens, new, 2, g, code, dtype, seed=g + 10).check()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_prompts(code, dtype):
    Case([300, 129, 700, 64], [300, 100, 257, 64], 2, 4, code, dtype, seed=3).check()


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("g", [1, 2, 3, 5, 6, 7, 8])
@pytest.mark.parametrize("n,length", [(128, 128), (33, 1000), (257, 1500), (600, 601)])
def test_prompts_of_odd_sizes_and_groups(code, g, n, length):
    Case([length, 17], [n, 9], 2, g, code, seed=g * n).check()


MODS = [dict(cap=20.0), dict(window=1), dict(window=64), dict(window=100), dict(prefix=True),
        dict(window=50, prefix=True), dict(slopes=True), dict(cap=5.0, slopes=True, window=333, prefix=True)]


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("mod", range(len(MODS)))
@pytest.mark.parametrize("new", [1, 6, 150])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_caps_biases_windows_and_prefixes(code, mod, new, dtype):
    m = dict(MODS[mod])
    lens = [1, 65, 200, 640, 1500]
    news = [min(n, new) for n in lens]
    c = Case(lens, news, 2, 3, code, dtype, seed=mod * 7 + new)
    if m.get("prefix"):
        m["prefix"] = [1, 0, 150, 333, 64]
    if m.get("slopes"):
        m["slopes"] = (2.0 ** -np.arange(1, 7)).tolist()
    c.check(**m)


def test_prefix_beyond_the_stored_tokens_and_below_zero():
    c = Case([100, 100], [40, 1], 1, 2, ref.INT8, seed=4)
    got = c.run(prefix=[1000, -5])
    out, tol = c.want(prefix=[100, 0])
    assert (np.abs(got.double().cpu().numpy() - out) <= tol).all()


@pytest.mark.parametrize("new", [1, 4, 200])
def test_strided_queries_and_given_output(new):
    c = Case([300, 400], [new, new], 2, 4, ref.E4M3, seed=5, fused=True)
    out = torch.full(tuple(c.q.shape), float("nan"), dtype=c.dtype, device="cuda")
    assert c.run(out=out) is out
    w, tol = c.want()
    assert (np.abs(out.double().cpu().numpy() - w) <= tol).all()


@pytest.mark.parametrize("new", [1, 5, 150])
@pytest.mark.parametrize("max_new", [1, 3, 64, 100000])
def test_a_wrong_max_new_costs_no_result(new, max_new):
    Case([260, 500], [new, new], 2, 4, ref.INT8, seed=6).check(max_new=max_new)


@pytest.mark.parametrize("new", [1, 5, 150])
def test_rows_behind_the_last_request_stay(new):
    c = Case([260, 500], [new, new], 2, 4, ref.INT8, seed=7, pad=7)
    out = torch.full(tuple(c.q.shape), 5.0, dtype=c.dtype, device="cuda")
    c.run(out=out)
    assert (out[2 * new:] == 5.0).all()
    w, tol = c.want()
    assert (np.abs(out[:2 * new].double().cpu().numpy() - w) <= tol).all()


@pytest.mark.parametrize("new", [4, 200])
@pytest.mark.parametrize("prefix", [False, True])
def test_queries_in_front_of_the_stored_tokens_get_zeros(new, prefix):
    """lens smaller than the number of queries: the first ones see nothing
    (or the prefix alone)."""
    c = Case([2, 90], [new, new], 2, 4, ref.INT8, seed=8)
    kw = dict(prefix=[1, 0]) if prefix else {}
    got = c.run(**kw).double().cpu().numpy()
    w, tol = c.want(**kw)
    assert (np.abs(got - w) <= tol).all()
    if not prefix:
        assert (got[:new - 2] == 0).all()


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 60, 2.0 ** 110])
@pytest.mark.parametrize("new", [4, 200])
def test_empty_rows_are_zeros_whatever_the_scales(new, scale):
    c = Case([2, 90], [new, new], 2, 4, ref.INT8, seed=27)
    c.vs *= np.float32(scale)
    got = c.run().double().cpu().numpy()
    assert (got[:new - 2] == 0).all() and np.isfinite(got).all()


@pytest.mark.parametrize("new", [1, 200])
def test_hidden_pages_of_tiny_values_beside_huge_ones(new):
    """Value scales 98 powers of two apart (a query's pages may be up to 2^100
    apart): what a row does not see must not count, however large 1 / scale is,
    and what it sees counts in the denominator with its weight."""
    c = Case([700], [new], 2, 4, ref.INT8, seed=28)
    c.vs[:] = np.float32(2.0 ** 60)
    c.vs[c.table[0, ::2]] = np.float32(2.0 ** -38)
    c.check(window=70)


@pytest.mark.parametrize("new", [1, 3, 130])
def test_requests_that_hold_nothing_get_zeros(new):
    c = Case([0, 200, 0], [new, new, new], 2, 4, ref.INT8, seed=9, extra_width=1)
    got = c.run().double().cpu().numpy()
    w, tol = c.want()
    assert (got[:new] == 0).all() and (got[2 * new:] == 0).all()
    assert (np.abs(got - w) <= tol).all()


@pytest.mark.parametrize("new", [1, 3, 130])
def test_pages_outside_the_pool_hide_their_tokens(new):
    c = Case([640, 300], [new, new], 2, 4, ref.E4M3, seed=12)
    bad = c.table.copy()
    bad[0, 3], bad[1, 0] = -1, 10 ** 6
    keep = c.table
    c.table = bad
    got = c.run().double().cpu().numpy()
    c.table = keep
    at = 0
    for b, hidden in ((0, range(192, 256)), (1, range(0, 64))):
        n = c.lens[b]
        q = c.q[at:at + new].double().cpu().numpy()
        k, v = rows_of(c.kc, c.ks, c.table[b], n, c.code), rows_of(c.vc, c.vs, c.table[b], n, c.code)
        on = ref.visible(n, new, 0, 0)
        on[:, list(hidden)] = False
        for h in range(c.heads):
            x = np.where(on, 128 ** -0.5 * q[:, h] @ k[:, h // c.g].T, -np.inf)
            w = np.exp(x - x.max(1, keepdims=True))
            w /= w.sum(1, keepdims=True)
            o, mass = w @ v[:, h // c.g], w @ np.abs(v[:, h // c.g])
            size = (128 ** -0.5 * np.abs(q[:, h]) @ np.abs(k[:, h // c.g]).T).max(1)[:, None]
            assert (np.abs(got[at:at + new, h] - o) <= bound(o, mass, size, c.dtype)).all()
        at += new


@pytest.mark.parametrize("new", [1, 130])
def test_lengths_beyond_the_table_are_cut(new):
    c = Case([128, 128], [new, new], 1, 4, ref.INT8, seed=13)
    if new > 128:
        c.new = [128, 128]
        c.q = c.q[:256].contiguous()
    got = c.run(lens=[10 ** 9, 128]).double().cpu().numpy()
    w, tol = c.want()
    assert (np.abs(got - w) <= tol).all()


@pytest.mark.parametrize("new", [1, 3, 130])
def test_stale_codes_behind_the_last_token_do_not_matter(new):
    """Recycled pages: whatever stands behind a request's last token, e4m3 NaN
    codes and infinite scales of other pages among it, is not read."""
    c = Case([70, 130], [min(new, 70), new], 2, 4, ref.E4M3, seed=14)
    for b, n in enumerate(c.lens):
        p = c.table[b, n // 64]
        c.kc[p, :, n % 64:] = 0x7f
        c.vc[p, :, n % 64:] = 0xff
    used = {int(x) for row in c.table for x in row if x >= 0}
    for p in set(range(c.kc.shape[0])) - used:
        c.ks[p], c.vs[p] = np.inf, np.nan
        c.kc[p], c.vc[p] = 0x7f, 0x7f
    c.check()


@pytest.mark.parametrize("new", [1, 130])
def test_value_scales_far_apart_and_blocks_of_zeros(new):
    c = Case([400, 640], [new, new], 2, 4, ref.INT8, seed=15)
    c.vs[::2] *= np.float32(2.0 ** -40)
    p = c.table[1, 2]
    c.vc[p], c.vs[p] = 0, 0
    c.kc[c.table[1, 5]], c.ks[c.table[1, 5]] = 0, 0
    c.check()


@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 90])
@pytest.mark.parametrize("new", [1, 130])
def test_values_very_small_and_very_large(scale, new):
    c = Case([400], [new], 2, 4, ref.INT8, seed=16)
    c.vs *= np.float32(scale)
    c.check()


@pytest.mark.parametrize("gain", [1e-30, 1e-3, 40.0, 1e20])
@pytest.mark.parametrize("new", [1, 130])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_queries_of_any_size(gain, new, dtype):
    """Large ones leave one key per row; both sides then take that key's value."""
    c = Case([333], [new], 2, 4, ref.INT8, dtype, seed=17)
    c.q = (c.q.float() * gain).to(c.dtype)
    got = c.run().double().cpu().numpy()
    out, tol = c.want()
    if gain <= 1:
        assert (np.abs(got - out) <= tol).all()
    else:
        at, _, size = 0, None, None
        q = c.q.double().cpu().numpy()
        k, v = rows_of(c.kc, c.ks, c.table[0], 333, c.code), rows_of(c.vc, c.vs, c.table[0], 333, c.code)
        on = ref.visible(333, new, 0, 0)
        for h in range(c.heads):
            x = np.where(on, 128 ** -0.5 * q[:, h] @ k[:, h // c.g].T, -np.inf)
            two = np.sort(x, 1)[:, -2:]
            size = (128 ** -0.5 * np.abs(q[:, h]) @ np.abs(k[:, h // c.g]).T).max(1)
            clear = (two[:, 1] - two[:, 0]) > 30 + 2.0 ** -15 * size   # one key carries the row
            pick = v[x.argmax(1), h // c.g]
            assert (np.abs(got[:, h] - pick)[clear] <= 2.0 ** -8 * np.abs(pick)[clear] + 1e-9).all()
        assert np.isfinite(got).all()


def test_nan_queries_stay_in_their_rows():
    for new in (1, 5, 150):
        c = Case([260, 500], [new, new], 2, 4, ref.INT8, seed=18)
        c.q[0, 3, 7] = float("nan")
        got = c.run().double().cpu().numpy()
        assert np.isnan(got[0, 3]).all()
        keep = torch.ones(c.q.shape[:2], dtype=torch.bool)
        keep[0, 3] = False
        c.q[0, 3, 7] = 0.0
        out, tol = c.want()
        k = keep.numpy()
        assert (np.abs(got - out) <= tol)[k].all()


@pytest.mark.parametrize("new", [1, 5, 150])
def test_the_same_call_gives_the_same_bits(new):
    c = Case([900, 2500, 64], [new, new, min(new, 64)], 2, 4, ref.E4M3, seed=19)
    a = c.run()
    for _ in range(3):
        assert torch.equal(a, c.run())


@pytest.mark.parametrize("new", [1, 5, 150])
def test_calls_on_several_streams_at_once(new):
    cases = [Case([700 + 100 * i, 90], [new, min(new, 90)], 2, 4, ref.INT8, seed=20 + i) for i in range(4)]
    for c in cases:
        c.store()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    outs = []
    for c, s in zip(cases, streams):
        with torch.cuda.stream(s):
            outs.append([c.run() for _ in range(3)])
    torch.cuda.synchronize()
    for c, o in zip(cases, outs):
        w, tol = c.want()
        for x in o:
            assert (np.abs(x.double().cpu().numpy() - w) <= tol).all()


def test_more_than_two_to_the_31_codes_in_the_pool():
    """Offsets past 32 bits: a request whose pages lie at both ends of a pool
    of 2.4e9 codes."""
    import online_rank_kv_b200 as ik
    pages, heads = 37000, 8
    shape = (pages, heads, 64, 128)
    k = torch.zeros(shape, dtype=torch.int8, device="cuda")
    v = torch.zeros(shape, dtype=torch.int8, device="cuda")
    ks, vs = torch.ones(pages, heads, device="cuda"), torch.ones(pages, heads, device="cuda")
    store = ik.Q8Pages.of(k, v, ks, vs)
    rows = torch.randn(2, 128, heads, 128, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    table = torch.tensor([[pages - 1, 0]], dtype=torch.int32, device="cuda")
    slots = torch.cat([torch.arange(64) + (pages - 1) * 64, torch.arange(64)]).to(torch.int32).cuda()
    store.append(rows[0], rows[1], slots)
    for n in (1, 100):
        q = torch.randn(n, heads * 2, 128, device="cuda").bfloat16()
        out = store.attention(q, table, torch.tensor([128], dtype=torch.int32, device="cuda"),
                              torch.tensor([0, n], dtype=torch.int32, device="cuda"), max_new=n)
        pg = [pages - 1, 0]
        kk = (k[pg].double() * ks[pg].double()[..., None, None]).permute(0, 2, 1, 3).reshape(128, heads, 128).cpu().numpy()
        vv = (v[pg].double() * vs[pg].double()[..., None, None]).permute(0, 2, 1, 3).reshape(128, heads, 128).cpu().numpy()
        o, mass, size = ref.attention(q.double().cpu().numpy(), kk, vv, 128 ** -0.5)
        assert (np.abs(out.double().cpu().numpy() - o) <= bound(o, mass, size, torch.bfloat16)).all()
    assert store.status() == 0


@pytest.mark.parametrize("code", CODES)
@pytest.mark.parametrize("new", [1, 5, 200])
@pytest.mark.parametrize("growth", [1.1, 1.7])
def test_scores_that_grow_along_the_keys(code, new, growth):
    """Each page's keys are larger than the last one's: the running maximum is
    raised again and again, by little and by much."""
    c = Case([900], [new], 2, 4, code, seed=21, gain=0.03)
    for j in range(15):
        c.ks[c.table[0, j]] = np.float32(2.0 ** -9 * growth ** j)
    c.check()


@pytest.mark.parametrize("new", [1, 200])
def test_scores_far_below_the_first_page(new):
    """A first page far above all others: their weights end below every range."""
    c = Case([900], [new], 2, 4, ref.INT8, seed=22)
    c.ks[c.table[0, 0]] *= np.float32(200.0)
    c.check()


@pytest.mark.parametrize("new", [1, 9, 40])
def test_many_requests_at_the_batch_limit(new):
    rng = np.random.default_rng(23)
    n = 8192 if new == 1 else 300
    lens = rng.integers(0 if new == 1 else new, 90, n).tolist()
    news = [min(k, new) for k in lens] if new == 1 else rng.integers(0, new + 1, n).tolist()
    Case(lens, news, 1, 2, ref.E4M3, seed=24).check()


@pytest.mark.parametrize("dtype,new", [("bf16", 1), ("f32", 6), ("bf16", 150)])
def test_buffers_that_are_16_byte_aligned_and_no_more(dtype, new):
    import ctypes
    import online_rank_kv_b200 as ik
    c = Case([700, 333], [new, new], 2, 4, ref.INT8, dtype, seed=25)
    n, per16 = c.q.shape[0], 16 // c.q.element_size()
    out = torch.zeros(c.q.numel() + per16, dtype=c.dtype, device="cuda")[per16:].view(c.q.shape)
    q = torch.zeros(c.q.numel() + per16, dtype=c.dtype, device="cuda")[per16:].view(c.q.shape).copy_(c.q)
    dt = ik.BF16 if dtype == "bf16" else ik.F32
    need = ik.LIB.iskv_q8_workspace(c.heads, 2, n, new, dt)
    ws = torch.empty(need + 16, dtype=torch.uint8, device="cuda")[16:]
    assert out.data_ptr() % 32 == 16 and ws.data_ptr() % 32 == 16
    table = torch.from_numpy(c.table.copy()).cuda()
    lens = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, new, 2 * new], dtype=torch.int32, device="cuda")
    store = c.store()
    a = ik._Q8Attention(2, table.shape[1], c.heads, dt, new, 0, 128 ** -0.5, 0.0, n, q.stride(0), q.data_ptr(),
                        out.data_ptr(), table.data_ptr(), lens.data_ptr(), cu.data_ptr(), None, None, ws.data_ptr(), need,
                        None)
    stream = torch.cuda.current_stream().cuda_stream
    assert ik.LIB.iskv_q8_attention(store._ref, ctypes.byref(a), stream) == 0
    w, tol = c.want()
    assert (np.abs(out.double().cpu().numpy() - w) <= tol).all()
    a.workspace_bytes = need - 1
    assert ik.LIB.iskv_q8_attention(store._ref, ctypes.byref(a), stream) == -2
    host = (ctypes.c_int32 * 4)()
    a.workspace_bytes, a.lens = need, ctypes.addressof(host)
    assert ik.LIB.iskv_q8_attention(store._ref, ctypes.byref(a), stream) == -1     # host memory


@pytest.mark.parametrize("new", [1, 150])
def test_a_stream_of_its_own_and_another_scale(new):
    c = Case([700, 333], [new, new], 2, 4, ref.INT8, seed=26)
    c.store()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = c.run(stream=s, scale=0.05)
    s.synchronize()
    w, tol = c.want(scale=0.05)
    assert (np.abs(got.double().cpu().numpy() - w) <= tol).all()


@pytest.mark.parametrize("max_new", [1, 300])
def test_no_queries_and_no_requests(max_new):
    import online_rank_kv_b200 as ik
    store = ik.Q8Pages(2, 2)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")
    out = store.attention(q, torch.zeros(3, 2, **i32), torch.zeros(3, **i32), torch.zeros(4, **i32), max_new=max_new)
    assert out.shape == (0, 8, 128)
    q = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device="cuda")
    given = torch.full_like(q, 3.0)
    out = store.attention(q, torch.zeros(0, 2, **i32), torch.zeros(0, **i32), torch.zeros(1, **i32), max_new=max_new, out=given)
    assert (out == 3.0).all()
    # requests without queries beside slots of a padded batch
    out = store.attention(q, torch.zeros(3, 2, **i32), torch.full((3,), 100, **i32), torch.zeros(4, **i32), max_new=max_new,
                          out=given)
    torch.cuda.synchronize()
    assert (out == 3.0).all() and store.status() == 0


def test_calls_in_turn_on_two_streams_by_argument():
    """Results and scratch memory of a call come from the stream it runs on:
    calls on two streams in turn, none waiting for the other, give what they
    give alone, and hold no memory of each other."""
    import online_rank_kv_b200 as ik
    cases = [Case([3000 + 700 * i, 90], [new, 1], 2, 4, ref.E4M3, seed=60 + i)
             for i, new in enumerate([1, 150, 5])]
    i32 = dict(dtype=torch.int32, device="cuda")
    args = []
    for c in cases:
        c.store()
        cu = np.concatenate([[0], np.cumsum(c.new)])
        args.append([torch.tensor(np.asarray(x), **i32) for x in (c.table, c.lens, cu)])
    def call(i, stream):
        table, lens, cu = args[i]
        return cases[i].store().attention(cases[i].q, table, lens, cu, max_new=max(cases[i].new), stream=stream)
    alone = [call(i, None) for i in range(3)]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = [(i, call(i, side if (k + i) % 2 else None)) for k in range(10) for i in range(3)]
    lens, add = torch.zeros(3, **i32), torch.full((3,), 70, **i32)
    table, free, n_free = torch.full((3, 2), -1, **i32), torch.arange(9, **i32), torch.full((1,), 9, **i32)
    torch.cuda.synchronize()
    plan = ik.page_plan(lens, add, table, free, n_free, tokens=211, stream=side)
    junk = [torch.full((8192,), 7, **i32) for _ in range(8)]     # the current stream goes on
    torch.cuda.synchronize()
    for i, o in outs:
        assert torch.equal(o, alone[i])
    assert plan.cu.tolist() == [0, 70, 140, 210] and plan.n_free.item() == 3 and plan.status.item() == 0
    assert all((j == 7).all() for j in junk)


@pytest.mark.parametrize("new", [1, 150])
def test_an_output_over_the_queries_is_refused(new):
    import online_rank_kv_b200 as ik
    c = Case([700, 333], [new, new], 2, 4, ref.INT8, seed=27)
    n = c.q.shape[0]
    both = torch.zeros(2 * n, c.heads, 128, dtype=c.dtype, device="cuda")
    both[:n] = c.q
    c.q = both[:n]
    for at in (0, 1, n - 1):
        with pytest.raises(ik.IskvError) as e:
            c.run(out=both[at:at + n])
        assert e.value.code == -1
    got = c.run(out=both[n:]).double().cpu().numpy()      # right behind them
    w, tol = c.want()
    assert (np.abs(got - w) <= tol).all()
