"""The paged 8-bit cache refuses bad arguments on the host, before any launch;
its binding's structures match the header; the reference's own pins.  No GPU."""

import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import paged_q8 as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _ik():
    import online_rank_kv_b200 as ik
    return ik


def _host(n=4096):
    """Host memory, 16-byte aligned: never a valid operand."""
    buf = (ctypes.c_char * (n + 16))()
    return buf, (ctypes.addressof(buf) + 15) // 16 * 16


def _store(ik, **kw):
    buf, at = _host()
    f = dict(pages=4, kv_heads=2, head_dim=128, page=64, code=0, k=at, v=at, k_scale=at, v_scale=at)
    f.update(kw)
    s = ik._Q8Pages(**f)
    s.keep = buf
    return s


@pytest.mark.parametrize("change,code", [
    (dict(pages=0), -1), (dict(pages=2 ** 25), -1), (dict(kv_heads=0), -1), (dict(code=2), -1), (dict(code=-1), -1),
    (dict(head_dim=64), -7), (dict(page=32), -7), (dict(kv_heads=65536), -7), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(k=8), -1), (dict(v_scale=2), -1), (dict(), -1)])
def test_both_calls_refuse_a_bad_store(change, code):
    ik = _ik()
    s = _store(ik, **change)
    _, at = _host()
    args = _attention(ik)
    assert ik.LIB.iskv_q8_attention(ctypes.byref(s), ctypes.byref(args), None) == code
    assert ik.LIB.iskv_q8_append(ctypes.byref(s), at, at, ik.BF16, 256, 256, 3, at, None, None) == code


def _attention(ik, **kw):
    buf, at = _host()
    f = dict(batch=2, width=3, q_heads=8, dtype=ik.BF16, max_new=1, window=0, scale=0.1, cap=0.0, tokens=2,
             q_stride=1024, q=at, out=at, table=at, lens=at, cu=at, prefix=None, slopes=None, workspace=at,
             workspace_bytes=1 << 40)
    f.update(kw)
    a = ik._Q8Attention(**f)
    a.keep = buf
    return a


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), -1), (dict(width=0), -1), (dict(width=2 ** 25), -1), (dict(q_heads=0), -1), (dict(q_heads=7), -1),
    (dict(q_heads=18), -7), (dict(batch=8193), -7), (dict(dtype=2), -1), (dict(max_new=0), -1), (dict(window=-1), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(cap=-1.0), -1), (dict(cap=float("nan")), -1), (dict(cap=float("inf")), -1), (dict(tokens=-1), -1),
    (dict(tokens=2 ** 31), -1), (dict(q=None), -1), (dict(out=None), -1), (dict(table=None), -1), (dict(lens=None), -1),
    (dict(cu=None), -1), (dict(workspace=None), -1), (dict(q_stride=1020), -1), (dict(q_stride=512), -1),
    (dict(q=24), -1), (dict(out=24), -1), (dict(workspace=24), -1), (dict(prefix=2), -1),
    (dict(batch=0), 0), (dict(tokens=0), 0), (dict(batch=0, q=None, table=None), 0), (dict(), -1)])
def test_attention_refuses_bad_arguments(change, code):
    ik = _ik()
    s, a = _store(ik), _attention(ik, **change)
    assert ik.LIB.iskv_q8_attention(ctypes.byref(s), ctypes.byref(a), None) == code
    assert ik.LIB.iskv_q8_attention(None, ctypes.byref(a), None) == -1
    assert ik.LIB.iskv_q8_attention(ctypes.byref(s), None, None) == -1


def test_append_refuses_bad_arguments():
    ik = _ik()
    s = _store(ik)
    buf, at = _host()

    def call(k=at, v=at, dt=ik.BF16, ks=256, vs=256, n=3, slots=at, status=None):
        return ik.LIB.iskv_q8_append(ctypes.byref(s), k, v, dt, ks, vs, n, slots, status, None)
    assert call() == -1                                   # host memory
    assert call(n=0) == 0 and call(n=0, k=None, slots=None) == 0
    for bad in (dict(k=None), dict(v=None), dict(slots=None), dict(dt=7), dict(n=-1), dict(n=2 ** 31), dict(ks=255),
                dict(vs=252), dict(ks=128), dict(dt=ik.F32, ks=258), dict(k=at + 8), dict(v=at + 2), dict(slots=at + 2),
                dict(status=at + 1)):
        assert call(**bad) == -1, bad
    assert ik.LIB.iskv_q8_append(None, at, at, 1, 256, 256, 3, at, None, None) == -1


@pytest.mark.parametrize("change,code", [
    (dict(batch=-1), -1), (dict(batch=8193), -7), (dict(width=0), -1), (dict(pages=0), -1), (dict(pages=2 ** 25), -1),
    (dict(width=2 ** 25), -1), (dict(tokens=-1), -1), (dict(lens=None), -1), (dict(add=None), -1), (dict(table=None), -1),
    (dict(free_pages=None), -1), (dict(n_free=None), -1), (dict(lens_out=None), -1), (dict(cu=None), -1),
    (dict(slots=None), -1), (dict(n_free_out=None), -1), (dict(status=None), -1), (dict(cu=6), -1), (dict(), -1)])
def test_page_plan_refuses_bad_arguments(change, code):
    ik = _ik()
    buf, at = _host()
    f = dict(batch=2, width=3, pages=4, tokens=2, lens=at, add=at, table=at, free_pages=at, n_free=at, lens_out=at,
             cu=at, slots=at, n_free_out=at, status=at)
    f.update(change)
    assert ik.LIB.iskv_page_plan(ctypes.byref(ik._PlanArgs(**f)), None) == code
    assert ik.LIB.iskv_page_plan(None, None) == -1


def test_workspace_sizes():
    ik = _ik()
    W = ik.LIB.iskv_q8_workspace
    for bad in ((0, 1, 1, 1, 1), (8, 0, 1, 1, 1), (7, 2, 1, 1, 1), (18, 2, 1, 1, 1), (8, 2, -1, 1, 1), (8, 2, 1, 0, 1),
                (8, 2, 1, 1, 5)):
        assert W(*bad) == -1
    assert 0 < W(8, 2, 1, 1, ik.BF16) <= W(8, 2, 1, 4, ik.BF16)
    assert W(32, 8, 0, 1, ik.F32) % 16 == 0


def test_the_binding_refuses_tensors_off_the_gpu_and_of_other_types():
    ik = _ik()
    z = torch.zeros(2, 1, 64, 128, dtype=torch.int8)
    s = torch.zeros(2, 1)
    with pytest.raises(ValueError):
        ik.Q8Pages.of(z, z, s, s)
    with pytest.raises(ValueError):
        ik.Q8Pages(2, 1, code=5)
    with pytest.raises(ValueError):
        i = torch.zeros(1, dtype=torch.int32)
        ik.page_plan(i, i, i.view(1, 1), i, i, tokens=1)


def test_structures_match_the_header(tmp_path):
    ik = _ik()
    structs = {"iskv_page_plan_args": ik._PlanArgs, "iskv_q8_pages": ik._Q8Pages,
               "iskv_q8_attention_args": ik._Q8Attention}
    lines = ['#include <stddef.h>', '#include <stdio.h>', '#include "iskv.h"', "int main(void) {"]
    for c, py in structs.items():
        lines.append(f'printf("{c} size %zu\\n", sizeof({c}));')
        lines += [f'printf("{c} {f} %zu\\n", offsetof({c}, {f}));' for f, _ in py._fields_]
    lines.append("return 0; }")
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    for line in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True, check=True).stdout.splitlines():
        c, f, v = line.split()
        assert int(v) == (ctypes.sizeof(structs[c]) if f == "size" else getattr(structs[c], f).offset), line


# ---- the reference itself ---------------------------------------------------
def test_reference_e4m3_codes_round_half_to_even_like_torch():
    x = np.random.default_rng(0).standard_normal(20000).astype(np.float32) * 100
    x = np.clip(x, -448, 448)
    ties = (ref._POSITIVE[:-1] + ref._POSITIVE[1:]) / 2
    x = np.concatenate([x, ties, -ties, ref._POSITIVE, x * 1e-4]).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(ref.e4m3_encode(x), want)


def test_reference_codes_are_within_half_a_step():
    g = np.random.default_rng(1)
    for code in (ref.INT8, ref.E4M3):
        codes = np.zeros((3, 2, 64, 128), dtype=np.int8 if code == ref.INT8 else np.uint8)
        scale = np.zeros((3, 2), dtype=np.float32)
        x = g.standard_normal((100, 2, 128)).astype(np.float32) * 5
        assert ref.append(codes, scale, x, list(range(64, 164)), code) == 0
        back = (ref.decode(codes, code) * scale[..., None, None])[1:].transpose(0, 2, 1, 3).reshape(128, 2, 128)[:100]
        s = np.repeat(scale[1:], 64, 0)[:100, :, None]
        step = s / 2 if code == ref.INT8 else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10)
        assert (np.abs(back - x) <= step * (1 + 1e-6)).all()


def test_reference_attention_is_softmax_attention():
    g = np.random.default_rng(2)
    q, k, v = g.standard_normal((5, 4, 128)), g.standard_normal((9, 2, 128)), g.standard_normal((9, 2, 128))
    out, _, _ = ref.attention(q, k, v, 0.1)
    for i in range(5):
        for h in range(4):
            w = np.exp(0.1 * k[:5 + i, h // 2] @ q[i, h])
            np.testing.assert_allclose(out[i, h], (w / w.sum()) @ v[:5 + i, h // 2], rtol=1e-12, atol=1e-13)


def test_reference_steps_keep_every_page_in_one_place():
    g = np.random.default_rng(3)
    lens, table = [0] * 5, np.full((5, 6), -1, dtype=np.int32)
    free, n = g.permutation(30).astype(np.int32), 30
    for _ in range(50):
        add = np.where(g.random(5) < 0.2, -1, np.minimum(g.integers(0, 90, 5), 6 * 64 - np.array(lens)))
        lens, cu, slots, n, status = ref.page_plan(lens, add, table, free, n, 500)
        assert status == 0 and cu[-1] == np.maximum(add, 0).sum()
        held = [int(table[b, j]) for b in range(5) for j in range(-(-lens[b] // 64))]
        assert sorted(held + free[:n].tolist()) == list(range(30))
