"""iskv_q8_attention against float64: single tokens, drafts and prompts over
ragged requests; masks, caps, distance biases, odd sizes, strides, bad pages,
inconsistent lengths, streams and captured graphs."""

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref
from q8_testlib import bound, random_store, rows_of, scattered_table, to_store

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
            bounds.append(bound(o, mass, size, self.dtype, cap, bias))
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
