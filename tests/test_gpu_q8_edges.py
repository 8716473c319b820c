"""iskv_q8_attention and iskv_q8_append at the edges of what they accept: work
lists past 2^31 steps, blocks of zeros, caps of any size, NaN, short lives of
inputs, waits that run out."""

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref
from q8_testlib import bound
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
