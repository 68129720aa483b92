"""CPU checks of the drafted-token calls: refusals before any CUDA call, malformed descriptors, the
frequency helper against its formulas, and the oracle's own pins. No device compute here."""
import ctypes
import importlib.util
import math
import os
import random
import subprocess
import sys
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_385_b200 as pa
from oracle import attention, tree
from tests.host_buffers import aligned_zeros
from tests.tree_case import TreeCase

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
cpu_only = pytest.mark.skipif(torch.cuda.is_available(), reason="host-pointer descriptors must never reach a GPU launch")
BF, F16, F32, I32, I64, E4 = (torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn)


def rope_args(**kw):
    T, hq, hkv, d, rot = 3, 4, 2, 128, 128
    a = {"q_out": aligned_zeros((T, hq, d), BF), "q": aligned_zeros((T, hq, d), BF), "key": aligned_zeros((T, hkv, d), BF),
         "value": aligned_zeros((T, hkv, d), BF), "positions": aligned_zeros((T,), I64),
         "inv_freq": aligned_zeros((rot // 2,), F32), "slots": aligned_zeros((T,), I64),
         "k_cache": aligned_zeros((4, hkv, 16, d), BF), "v_cache": aligned_zeros((4, hkv, 16, d), BF)}
    return {**a, **kw}


def tree_args(**kw):
    T, hq, hkv, d = 5, 4, 2, 128
    a = {"out": aligned_zeros((T, hq, d), BF), "q": aligned_zeros((T, hq, d), BF),
         "k_cache": aligned_zeros((8, hkv, 16, d), BF), "v_cache": aligned_zeros((8, hkv, 16, d), BF),
         "bt": aligned_zeros((2, 4), I32), "start": aligned_zeros((3,), I32), "lens": aligned_zeros((2,), I32),
         "mask": aligned_zeros((T, 1), I64)}
    return {**a, **kw}


def commit_args(**kw):
    a = {"k_cache": aligned_zeros((8, 2, 16, 128), BF), "v_cache": aligned_zeros((8, 2, 16, 128), BF),
         "bt": aligned_zeros((2, 4), I32), "start": aligned_zeros((3,), I32), "lens": aligned_zeros((2,), I32),
         "accepted": aligned_zeros((2, 3), I32), "accepted_lens": aligned_zeros((2,), I32), "new": aligned_zeros((2,), I32)}
    return {**a, **kw}


def refs(args):
    return [None if t is None else ctypes.byref(t if isinstance(t, pa.PaTensor) else pa.as_pa_tensor(t, n, device=False))
            for n, t in args.items()]


def rope(args, **kw):
    o = pa.PaRopeOpts()
    pa.lib().pa_rope_opts_init(ctypes.byref(o))
    for k, v in kw.items():
        setattr(o, k, v)
    return pa.lib().pa_rope_and_cache(*refs(args), ctypes.byref(o), None)


def attend(args, n=5, scale=0.1, cap=0.0, hkv=2, **kw):
    o = pa.PaDecodeOpts()
    pa.lib().pa_decode_opts_init(ctypes.byref(o))
    for k, v in kw.items():
        setattr(o, k, v)
    return pa.lib().pa_decode_tree(*refs(args), n, scale, cap, hkv, ctypes.byref(o), None)


def commit(args):
    return pa.lib().pa_commit_tree(*refs(args), None, None)


def shifted(shape, dtype, by):
    """A tensor whose data starts `by` bytes past an aligned boundary."""
    n = int(np.prod(shape)) * torch.tensor([], dtype=dtype).element_size()
    return aligned_zeros((n + 256,), torch.uint8)[by:by + n].view(dtype).view(*shape)


INVALID, UNSUPPORTED = pa.PA_ERR_INVALID_ARG, pa.PA_ERR_UNSUPPORTED


@cpu_only
@pytest.mark.parametrize("change,status,said", [
    ({"key": None}, INVALID, "key is NULL"),
    ({"q": None}, INVALID, "together"),
    ({"q_out": aligned_zeros((3, 2, 128), BF)}, INVALID, "q_out shape"),
    ({"q": aligned_zeros((3, 4, 128), F16)}, INVALID, "dtype"),
    ({"q": aligned_zeros((2, 4, 128), BF), "q_out": aligned_zeros((2, 4, 128), BF)}, INVALID, "num_tokens"),
    ({"value": aligned_zeros((3, 1, 128), BF)}, INVALID, "value shape"),
    ({"positions": aligned_zeros((3,), I32)}, INVALID, "positions"),
    ({"positions": aligned_zeros((4,), I64)}, INVALID, "positions"),
    ({"positions": aligned_zeros((6,), I64)[::2]}, INVALID, "contiguous"),
    ({"slots": aligned_zeros((3,), I32)}, INVALID, "slot_mapping"),
    ({"inv_freq": aligned_zeros((64,), F16)}, INVALID, "inv_freq"),
    ({"inv_freq": aligned_zeros((68,), F32)}, INVALID, "inv_freq"),
    ({"inv_freq": aligned_zeros((0,), F32)}, INVALID, "inv_freq"),
    ({"inv_freq": aligned_zeros((6,), F32)}, UNSUPPORTED, "multiple of 8"),
    ({"inv_freq": aligned_zeros((128,), F32)[::2]}, INVALID, "inv_freq must be contiguous"),
    ({"k_cache": aligned_zeros((4, 2, 16, 128), E4)}, INVALID, "dtypes differ"),
    ({"k_cache": aligned_zeros((4, 2, 16, 128), F16), "v_cache": aligned_zeros((4, 2, 16, 128), F16)}, INVALID, "does not match"),
    ({"k_cache": aligned_zeros((4, 2, 16, 64), BF), "v_cache": aligned_zeros((4, 2, 16, 64), BF)}, INVALID, "cache shape"),
    ({"key": shifted((3, 2, 128), BF, 8)}, INVALID, "aligned"),
    ({"q_out": aligned_zeros((3, 4, 129), BF)[..., :128]}, INVALID, "aligned"),
])
def test_rope_refusals(change, status, said):
    assert rope(rope_args(**change)) == status
    assert said in pa.pa_last_error()


@cpu_only
def test_rope_option_refusals_and_empty_calls():
    e4 = {"k_cache": aligned_zeros((4, 2, 16, 128), E4), "v_cache": aligned_zeros((4, 2, 16, 128), E4)}
    assert rope(rope_args(**e4), k_scale=0.0) == INVALID and rope(rope_args(**e4), v_scale=float("inf")) == INVALID
    assert rope(rope_args(), magnitude=float("nan")) == INVALID
    big = {n: aligned_zeros((1, 1, 520), BF) for n in ("q_out", "q", "key", "value")}
    big |= {n: aligned_zeros((1,), I64) for n in ("positions", "slots")}
    big |= {n: aligned_zeros((1, 1, 16, 520), BF) for n in ("k_cache", "v_cache")}
    assert rope(rope_args(**big)) == UNSUPPORTED
    none = {n: aligned_zeros((0, h, 128), BF) for n, h in (("q_out", 4), ("q", 4), ("key", 2), ("value", 2))}
    assert rope(rope_args(**none, positions=aligned_zeros((0,), I64), slots=aligned_zeros((0,), I64))) == pa.PA_OK
    # What is right gets as far as the device (there is none here).
    assert rope(rope_args()) == pa.PA_ERR_CUDA and rope(rope_args(q=None, q_out=None)) == pa.PA_ERR_CUDA


@cpu_only
@pytest.mark.parametrize("change,status,said", [
    ({"out": None}, INVALID, "out is NULL"),
    ({"out": aligned_zeros((5, 4, 128), F16)}, INVALID, "out dtype"),
    ({"out": aligned_zeros((4, 4, 128), BF)}, INVALID, "out shape"),
    ({"k_cache": aligned_zeros((8, 2, 16, 128), E4)}, INVALID, "dtypes differ"),
    ({"k_cache": aligned_zeros((8, 2, 16, 128), F16), "v_cache": aligned_zeros((8, 2, 16, 128), F16)}, INVALID, "needs"),
    ({"k_cache": aligned_zeros((8, 3, 16, 128), BF), "v_cache": aligned_zeros((8, 3, 16, 128), BF)}, INVALID, "num_kv_heads"),
    ({"k_cache": aligned_zeros((0, 2, 16, 128), BF), "v_cache": aligned_zeros((0, 2, 16, 128), BF)}, INVALID, "empty pool"),
    ({"start": aligned_zeros((2,), I32)}, INVALID, "query_start"),
    ({"lens": aligned_zeros((2,), I64)}, INVALID, "context_lens"),
    ({"bt": aligned_zeros((2, 0), I32)}, INVALID, "columns"),
    ({"bt": aligned_zeros((2, 4), I64)}, INVALID, "block_tables"),
    ({"mask": aligned_zeros((5, 1), I32)}, INVALID, "tree_mask"),
    ({"mask": aligned_zeros((4, 1), I64)}, INVALID, "tree_mask"),
    ({"mask": aligned_zeros((5, 2), I64)[:, :1]}, INVALID, "tree_mask"),
    ({"mask": aligned_zeros((5, 5), I64)}, UNSUPPORTED, "words"),
    ({"q": shifted((5, 4, 128), BF, 8)}, INVALID, "aligned"),
    ({"k_cache": shifted((8, 2, 16, 128), BF, 16)}, INVALID, "128-byte"),
])
def test_tree_refusals(change, status, said):
    assert attend(tree_args(**change)) == status
    assert said in pa.pa_last_error()


@cpu_only
def test_tree_option_refusals_and_empty_calls():
    for kw in ({"n": 0}, {"n": -1}, {"scale": float("nan")}, {"cap": -1.0}, {"cap": float("inf")}, {"max_context_len": -1},
               {"partition_tokens": 16}, {"kernel": 0}, {"prefix_kernel": 1}, {"hkv": 3}, {"hkv": 0}):
        assert attend(tree_args(), **kw) == INVALID, kw
    assert attend(tree_args(), n=65) == UNSUPPORTED and attend(tree_args(mask=None), n=257) == UNSUPPORTED
    for hq, hkv, d, dt in ((17, 1, 128, BF), (4, 2, 96, BF), (4, 2, 64, E4)):
        a = tree_args(out=aligned_zeros((5, hq, d), BF), q=aligned_zeros((5, hq, d), BF),
                      k_cache=aligned_zeros((8, hkv, 16, d), dt), v_cache=aligned_zeros((8, hkv, 16, d), dt))
        assert attend(a, hkv=hkv) == UNSUPPORTED, (hq, hkv, d, dt)
    e4 = tree_args(k_cache=aligned_zeros((8, 2, 16, 128), E4), v_cache=aligned_zeros((8, 2, 16, 128), E4))
    assert attend(e4, k_scale=0.0) == INVALID
    held = tree_args()
    mask = pa.as_pa_tensor(held["mask"], "mask", device=False)
    mask.data += 4
    assert attend({**held, "mask": mask}) == INVALID and "8-byte" in pa.pa_last_error()
    empty = tree_args(out=aligned_zeros((0, 4, 128), BF), q=aligned_zeros((0, 4, 128), BF), mask=aligned_zeros((0, 1), I64))
    assert attend(empty) == pa.PA_OK
    assert attend(tree_args()) == pa.PA_ERR_CUDA and attend(tree_args(mask=None)) == pa.PA_ERR_CUDA


@cpu_only
def test_tree_workspace():
    """A table wide enough for split contexts needs the workspace that the sizing call names, 256-byte aligned."""
    need = pa.pa_decode_tree_workspace_bytes(2, 4, 2, 128, 5, 16 * 4096)
    assert need > 0 and need % 256 == 0
    assert pa.pa_decode_tree_workspace_bytes(2, 4, 2, 128, 5, 64) == 0  # one key block: nothing to split
    assert pa.pa_decode_tree_workspace_bytes(0, 4, 2, 128, 5, 4096) == 0
    r = random.Random(0)  # sized once for the largest, it does for every smaller call
    for _ in range(300):
        group, hkv, d = r.choice([1, 3, 4, 8, 16]), r.choice([1, 8, 32]), r.choice([64, 128])
        b, n, c = r.randint(1, 300), r.randint(1, 256), r.choice([60, 129, 250, 260, 3000, 131072])
        most = pa.pa_decode_tree_workspace_bytes(b, group * hkv, hkv, d, n, c)
        for _ in range(5):
            less = pa.pa_decode_tree_workspace_bytes(r.randint(1, b), group * hkv, hkv, d, r.randint(1, n), r.randint(1, c))
            assert less <= most, (b, group, hkv, d, n, c)
    a = tree_args(bt=aligned_zeros((2, 4096), I32))
    ws = aligned_zeros((need + 256,), torch.uint8)
    assert attend(a) == pa.PA_ERR_WORKSPACE
    assert attend(a, workspace=ws.data_ptr(), workspace_bytes=need - 1) == pa.PA_ERR_WORKSPACE
    assert attend(a, workspace=ws.data_ptr() + 128, workspace_bytes=need) == INVALID
    assert attend(a, workspace=ws.data_ptr(), workspace_bytes=need) == pa.PA_ERR_CUDA
    assert attend(a, max_context_len=64) == pa.PA_ERR_CUDA


@cpu_only
@pytest.mark.parametrize("change,status,said", [
    ({"k_cache": None}, INVALID, "k_cache is NULL"),
    ({"k_cache": aligned_zeros((8, 2, 16, 128), F32), "v_cache": aligned_zeros((8, 2, 16, 128), F32)}, INVALID, "dtype"),
    ({"v_cache": aligned_zeros((8, 2, 16, 64), BF)}, INVALID, "shape"),
    ({"k_cache": aligned_zeros((8, 2, 16, 4), BF), "v_cache": aligned_zeros((8, 2, 16, 4), BF)}, UNSUPPORTED, "16"),
    ({"accepted": aligned_zeros((2, 3), I64)}, INVALID, "accepted"),
    ({"accepted": aligned_zeros((2, 6), I32)[:, ::2]}, INVALID, "accepted"),
    ({"accepted_lens": aligned_zeros((3,), I32)}, INVALID, "accepted_lens"),
    ({"new": aligned_zeros((2,), I64)}, INVALID, "new_context_lens"),
    ({"start": aligned_zeros((4,), I32)}, INVALID, "query_start"),
    ({"bt": aligned_zeros((2, 0), I32)}, INVALID, "columns"),
])
def test_commit_refusals(change, status, said):
    assert commit(commit_args(**change)) == status
    assert said in pa.pa_last_error()


@cpu_only
def test_commit_overlaps_and_empty_calls():
    lens = aligned_zeros((4,), I32)
    for new in (lens[:2], lens[1:3]):
        assert commit(commit_args(lens=lens[:2], new=new)) == INVALID and "overlaps" in pa.pa_last_error()
    assert commit(commit_args(lens=lens[:2], new=lens[2:])) == pa.PA_ERR_CUDA
    assert commit(commit_args(new=None)) == pa.PA_ERR_CUDA
    empty = commit_args(bt=aligned_zeros((0, 4), I32), start=aligned_zeros((1,), I32),
                        **{n: aligned_zeros((0,), I32) for n in ("lens", "accepted_lens", "new")},
                        accepted=aligned_zeros((0, 3), I32))
    assert commit(empty) == pa.PA_OK


def moved(args, name, by):
    """args with one tensor's data moved by some bytes."""
    t = pa.as_pa_tensor(args[name], name, device=False)
    t.data += by
    return {**args, name: t}


@cpu_only
@pytest.mark.parametrize("make,call,names", [
    (rope_args, rope, ("positions", "inv_freq", "slots")), (tree_args, attend, ("bt", "start", "lens")),
    (commit_args, commit, ("bt", "start", "lens", "accepted", "accepted_lens", "new"))])
def test_unaligned_index_tensors_are_refused(make, call, names):
    held = make()
    for name in names:
        for by in (1, 2, 3):
            assert call(moved(held, name, by)) == INVALID and "aligned" in pa.pa_last_error(), name
    if call is commit:
        return
    word = aligned_zeros((2,), I32)
    assert call(held, error_word=word.data_ptr() + 2) == INVALID and "aligned" in pa.pa_last_error()
    assert call(held, error_word=word.data_ptr()) == pa.PA_ERR_CUDA


@cpu_only
def test_pairs_in_one_place():
    """Queries may be worked on in place, with their own strides; commit's two pools may not be one."""
    wide = aligned_zeros((5, 4, 256), BF)[..., :128]
    tight = wide.as_strided((5, 4, 128), (512, 128, 1))
    assert attend(tree_args(out=wide, q=wide)) == pa.PA_ERR_CUDA
    assert attend(tree_args(out=wide, q=tight)) == INVALID and "in place" in pa.pa_last_error()
    assert rope(rope_args(q=wide[:3], q_out=wide[:3])) == pa.PA_ERR_CUDA
    assert rope(rope_args(q=wide[:3], q_out=tight[:3])) == INVALID and "in place" in pa.pa_last_error()
    pools = aligned_zeros((2, 8, 2, 16, 128), BF)
    assert commit(commit_args(k_cache=pools[0], v_cache=pools[1])) == pa.PA_ERR_CUDA
    assert commit(commit_args(k_cache=pools[0], v_cache=pools[0])) == INVALID and "overlap" in pa.pa_last_error()
    both = aligned_zeros((9, 2, 16, 128), BF)
    assert commit(commit_args(k_cache=both[:8], v_cache=both[1:])) == INVALID


@cpu_only
def test_scales_and_caps_out_of_range():
    assert attend(tree_args(), scale=3e38) == INVALID and "overflows" in pa.pa_last_error()
    e4 = tree_args(k_cache=aligned_zeros((8, 2, 16, 128), E4), v_cache=aligned_zeros((8, 2, 16, 128), E4))
    assert attend(e4, scale=1e20, k_scale=1e20) == INVALID
    assert attend(tree_args(), cap=1024.5) == UNSUPPORTED and "1024" in pa.pa_last_error()
    assert attend(tree_args(), cap=1024.0) == pa.PA_ERR_CUDA


@cpu_only
def test_injected_failures():
    try:
        for call in (lambda: rope(rope_args()), lambda: attend(tree_args()), lambda: commit(commit_args())):
            pa.pa_debug_fail_next_launches(1)
            assert call() == pa.PA_ERR_CUDA and "injected" in pa.pa_last_error()
    finally:
        pa.pa_debug_fail_next_launches(0)


@cpu_only
@pytest.mark.parametrize("seed", range(3))
def test_malformed_descriptors_return_a_status(seed):
    r = random.Random(seed)
    extremes = [0, 1, -1, 2, 3, 17, 65536, (1 << 31) - 1, 1 << 31, 1 << 40, 1 << 62, -(1 << 62)]
    statuses = {pa.PA_OK, INVALID, UNSUPPORTED, pa.PA_ERR_WORKSPACE, pa.PA_ERR_CUDA}
    seen = set()
    for _ in range(4000):
        make, call = r.choice([(rope_args, rope), (tree_args, attend), (commit_args, commit)])
        held = make()
        ts = {n: pa.as_pa_tensor(t, n, device=False) for n, t in held.items()}
        for _ in range(r.choice([0, 1, 1, 2, 3])):
            t = r.choice(list(ts.values()))
            k = r.randrange(5)
            if k == 0:
                t.dtype = r.randrange(-1, 8)
            elif k == 1:
                t.shape[r.randrange(4)] = r.choice(extremes)
            elif k == 2:
                t.stride[r.randrange(4)] = r.choice(extremes + [8, 128])
            elif k == 3:
                t.data = r.choice([0, (t.data or 0) + 2, (t.data or 0) + 8])
            else:
                t.ndim = r.randint(-1, 5)
        kw = {}
        if call is attend:
            kw = {"n": r.choice([5, 0, 64, 65, 1 << 30]), "hkv": r.choice([2, 2, ts["k_cache"].shape[1] & 0x7fffffff]),
                  "max_context_len": r.choice([0, 1, 64, (1 << 31) - 1])}
        status = call(ts, **kw)
        assert status in statuses
        seen.add(status)
    assert {INVALID, pa.PA_ERR_CUDA} <= seen
    assert pa.pa_decode_tree_workspace_bytes(65535, 1 << 20, 65535, 128, 256, (1 << 31) - 1) > 0


def test_rope_opts_layout(tmp_path):
    fields = [n for n, _ in pa.PaRopeOpts._fields_]
    src = tmp_path / "o.c"
    src.write_text('#include <stdio.h>\n#include "pa.h"\nint main(void) {\n  printf("%zu\\n", sizeof(pa_rope_opts));\n' +
                   "".join(f'  printf("%zu\\n", offsetof(pa_rope_opts, {n}));\n' for n in fields) + "  return 0;\n}\n")
    exe = str(tmp_path / "o")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", exe], check=True)
    got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [ctypes.sizeof(pa.PaRopeOpts)] + [getattr(pa.PaRopeOpts, n).offset for n in fields]
    packed = pa.PaRopeOpts.from_buffer_copy(pa._ROPE_OPTS.pack(True, 1.5, 0.25, 0.5, 1 << 40))
    assert [getattr(packed, n) for n in fields] == [1, 1.5, 0.25, 0.5, 1 << 40]


def test_frequencies():
    """Each kind's formula in Python floats; the library rounds its float64 once, so one float32 step at most."""
    def near(got, want):
        assert got.dtype == torch.float32 and len(got) == len(want)
        assert all(abs(float(g) - w) <= 2.0 ** -24 * w * (1 + 1e-6) for g, w in zip(got, want))

    R, base, L, f = 128, 500000.0, 8192, 8.0
    theta = [base ** (-2 * i / R) for i in range(R // 2)]
    near(pa.pa_rope_inv_freq(R, base), theta)
    near(pa.pa_rope_inv_freq(R, base, pa.PA_ROPE_LINEAR, f), [t / f for t in theta])
    near(pa.pa_rope_inv_freq(R, base, pa.PA_ROPE_BASE, f), [(base * f ** (R / (R - 2))) ** (-2 * i / R) for i in range(R // 2)])

    def blend(t, keep):
        keep = min(1.0, max(0.0, keep))
        return t * keep + t / f * (1 - keep)

    turns = [L * t / (2 * math.pi) for t in theta]
    near(pa.pa_rope_inv_freq(R, base, pa.PA_ROPE_BANDS, f, L, 1.0, 4.0), [blend(t, (w - 1) / 3) for t, w in zip(theta, turns)])

    def index(w):
        return R * math.log(L / (w * 2 * math.pi)) / (2 * math.log(base))

    lo, hi = math.floor(index(32)), math.ceil(index(1))
    assert 0 < lo < hi < R // 2
    near(pa.pa_rope_inv_freq(R, base, pa.PA_ROPE_RAMP, f, L, 1.0, 32.0), [blend(t, 1 - (i - lo) / (hi - lo)) for i, t in enumerate(theta)])
    # The fastest pairs keep their frequency and the slowest take the scaled one.
    ramp = pa.pa_rope_inv_freq(R, base, pa.PA_ROPE_RAMP, f, L, 1.0, 32.0)
    assert float(ramp[0]) == 1.0 and abs(float(ramp[-1]) * f / theta[-1] - 1) < 2.0 ** -23
    slow = pa.pa_rope_inv_freq(R, base, pa.PA_ROPE_BASE, f)
    assert float(slow[0]) == 1.0 and abs(float(slow[-1]) * f / theta[-1] - 1) < 2.0 ** -22


@pytest.mark.parametrize("args", [(0,), (7,), (64, 1.0), (64, float("nan")), (64, 1e4, 9), (64, 1e4, 1, 0.5), (2, 1e4, 2, 2.0),
                                  (64, 1e4, 3, 2.0, 0), (64, 1e4, 3, 2.0, 100, 4.0, 4.0), (64, 1e4, 4, 2.0, 100, 0.0, 4.0)])
def test_frequency_refusals(args):
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.pa_rope_inv_freq(*args)
    assert e.value.status == INVALID


def test_binding_refuses_host_tensors():
    a = rope_args()
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_rope_and_cache(*a.values())
    t = tree_args()
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_decode_tree(*list(t.values()), 5, 0.1, 2)
    with pytest.raises(TypeError, match="not both"):
        pa.pa_decode_tree(*list(t.values()), 5, 0.1, 2, opts=pa.PaDecodeOpts(), k_scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pa.pa_commit_tree(*commit_args().values())
    for call, a, name in ((pa.pa_rope_and_cache, rope_args(key=None), "key"), (pa.pa_commit_tree, commit_args(lens=None), "context_lens")):
        with pytest.raises(ValueError, match="CUDA|" + name):
            call(*a.values())


def test_views_of_tensors():
    """The extension's views are as_pa_tensor's, field by field; what is no view is named by its place."""
    ts = (torch.zeros(3, 4, 8)[:, 1:3], None, torch.zeros(5, dtype=I64), torch.zeros(0, 2, dtype=BF), torch.tensor(1, dtype=I32),
          torch.zeros(2, 3, 4, 5, dtype=F16).permute(3, 0, 2, 1), torch.zeros(2, 6, dtype=E4))
    keep, refs_ = pa._views.pack(ts, pa._DTYPES, -1)
    assert refs_[1] is None and len(refs_) == len(ts)
    for t, at in zip(ts, refs_):
        if t is not None:
            got, want = pa.PaTensor.from_address(at), pa.as_pa_tensor(t, "t", device=False)
            assert bytes(got) == bytes(want)
    assert pa._views.pack((ts[0], torch.zeros(1, dtype=torch.uint8)), pa._DTYPES, -1) == 1
    assert pa._views.pack((torch.zeros(1, 1, 1, 1, 1),), pa._DTYPES, -1) == 0
    assert pa._views.pack((ts[0],), pa._DTYPES, 0) == 0  # on another device
    for bad in ((None, pa._DTYPES, 0), ((3,), pa._DTYPES, 0), ((ts[0],), [], 0), ((ts[0],), pa._DTYPES, "0")):
        with pytest.raises((TypeError, AttributeError)):
            pa._views.pack(*bad)


# ---- the oracle's own pins -------------------------------------------------------------------------


def test_oracle_chain_is_prefill_and_one_node_is_decode():
    c = TreeCase("bf16", 64, 2, 2, [5, 9], [40, 9], masks=None, seed=1)
    got, weight = c.oracle()
    pools = (c.host_pool(0), c.host_pool(1))
    q = c.q_host.double().numpy()
    want = attention.prefill_paged(q, *pools, c.bt_host.numpy(), c.start_host, c.lens_host, c.scale, 2, "bf16")
    assert np.abs(got - want).max() < 1e-13 and np.all(weight >= np.abs(got) - 1e-13)
    c = TreeCase("f16", 64, 2, 2, [1, 1], [40, 9], seed=2)
    want = attention.decode_paged(c.q_host.double().numpy(), c.host_pool(0), c.host_pool(1), c.bt_host.numpy(), c.lens_host,
                                  c.scale, 2, "f16")
    assert np.abs(c.oracle()[0] - want).max() < 1e-13


def test_oracle_mask_and_cap_against_loops():
    c = TreeCase("f16", 64, 1, 1, [4], [6], masks=[0b0001, 0b0011, 0b0101, 0], softcap=1.5, seed=3)
    c.lens_host = [6]
    got, _ = c.oracle()
    K, V = (attention.gather_context(c.host_pool(i), c.bt_host.numpy()[0], 6, 0, "f16") for i in (0, 1))
    for i, sees in enumerate(([0, 1, 2], [0, 1, 2, 3], [0, 1, 2, 4], [0, 1])):
        x = [1.5 * math.tanh(c.scale * math.fsum(a * b for a, b in zip(c.q_host[i, 0].tolist(), K[t].tolist())) / 1.5) for t in sees]
        w = [math.exp(v) for v in x]
        want = [math.fsum(a * V[t][d] for a, t in zip(w, sees)) / math.fsum(w) for d in range(64)]
        assert np.abs(got[i, 0] - want).max() < 1e-12


@pytest.mark.parametrize("pairs", [False, True])
def test_oracle_rotation_is_complex_multiplication(pairs):
    r = np.random.default_rng(4)
    x, pos, inv = r.standard_normal((5, 2, 24)), np.array([0, 1, -3, 1000, 10 ** 6]), r.random(8).astype(np.float32)
    got = tree.rotate(x, pos, inv, pairs, 1.5)
    a, b = (x[..., 0:16:2], x[..., 1:16:2]) if pairs else (x[..., :8], x[..., 8:16])
    z = 1.5 * (a + 1j * b) * np.exp(1j * pos[:, None, None] * inv.astype(np.float64))
    u, v = (got[..., 0:16:2], got[..., 1:16:2]) if pairs else (got[..., :8], got[..., 8:16])
    assert np.abs(u - z.real).max() < 1e-12 and np.abs(v - z.imag).max() < 1e-12
    assert np.array_equal(got[..., 16:], x[..., 16:])


def test_planted_mistakes_are_seen():
    """The bound of the GPU tests is narrow enough: an oracle with a mistake in it falls outside."""
    c = TreeCase("bf16", 128, 1, 4, [9], [40], seed=5)
    want, weight = c.oracle()
    right = c.masks
    for wrong in ([m | 1 << 8 for m in right], [m >> 1 for m in right], None):
        c.masks = wrong
        assert (np.abs(c.oracle()[0] - want) > c.bound(want, weight)).any()
    c.masks = right
    c.softcap = 30.0
    assert (np.abs(c.oracle()[0] - want) > c.bound(want, weight)).any()


# ---- sizing over models of fewer heads --------------------------------------------------------------


@cpu_only
def test_tree_workspace_does_for_smaller_models():
    """What is named for the largest sizes does for every call of fewer heads of either kind too: a smaller group
    takes a form with more spans, fewer KV heads one with longer tiles."""
    size = pa.pa_decode_tree_workspace_bytes
    assert size(64, 64, 8, 128, 1, 8192) <= size(64, 128, 8, 128, 1, 8192)
    assert size(64, 32, 8, 128, 8, 8192) <= size(64, 32, 32, 128, 8, 8192)
    r = random.Random(1)
    for _ in range(400):
        hkv, hq = r.choice([1, 2, 7, 8, 32, 100]), 0
        hq = hkv * r.choice([1, 2, 3, 4, 8, 16])
        b, n, c = r.choice([1, 2, 9, r.randint(1, 300)]), r.choice([1, 2, r.randint(1, 256)]), r.choice([60, 129, 250, 260, 321, 3000, 131072])
        most = size(b, hq, hkv, 128, n, c)
        for _ in range(12):
            less_kv = r.randint(1, hkv)
            group = r.randint(1, min(16, hq // less_kv))
            less = (r.randint(1, b), group * less_kv, less_kv, 128, r.choice([n, r.randint(1, n)]), r.choice([c, r.randint(1, c)]))
            assert size(*less) <= most, ((b, hq, hkv, 128, n, c), less)
    # A call takes the workspace of a larger model.
    for hq, hkv, n in ((4, 2, 5), (16, 1, 1), (3, 3, 17), (16, 1, 9), (4, 4, 64), (8, 1, 64)):
        ws = aligned_zeros((size(2, 64, 8, 128, 64, 16 * 4096),), torch.uint8)
        T = 2 * n
        a = tree_args(out=aligned_zeros((T, hq, 128), BF), q=aligned_zeros((T, hq, 128), BF), mask=None,
                      k_cache=aligned_zeros((8, hkv, 16, 128), BF), v_cache=aligned_zeros((8, hkv, 16, 128), BF),
                      bt=aligned_zeros((2, 4096), I32))
        assert attend(a, n=n, hkv=hkv, workspace=ws.data_ptr(), workspace_bytes=ws.numel()) == pa.PA_ERR_CUDA, pa.pa_last_error()


# ---- the binding without its extension ---------------------------------------------------------------


def test_import_without_the_views_extension():
    """The package needs the library alone: without _views the calls marshal their tensors in Python."""
    code = ("import sys\nsys.modules['paged_kv_cache_385_b200._views'] = None\n"
            "import torch, paged_kv_cache_385_b200 as pa\nassert pa._views is None\n"
            "x = torch.zeros(1, dtype=torch.int32)\n"
            "try:\n    pa.pa_commit_tree(x, x, x, x, x, x, x)\n"
            "except ValueError as e:\n    assert 'k_cache must be a CUDA tensor' in str(e), e\n"
            "else:\n    raise AssertionError\nprint(pa.pa_version())\n")
    got = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, cwd=ROOT)
    assert got.returncode == 0 and got.stdout.strip() == pa.pa_version(), got.stderr


def test_views_in_python_are_the_extensions():
    ts = (torch.zeros(3, 4, 8)[:, 1:3], None, torch.zeros(0, 2, dtype=BF), torch.tensor(1, dtype=I32),
          torch.zeros(2, 3, 4, 5, dtype=F16).permute(3, 0, 2, 1), torch.zeros(2, 6, dtype=E4))
    bad = ((ts[0], torch.zeros(1, dtype=torch.uint8)), (torch.zeros(1, 1, 1, 1, 1),))
    with_ext, in_python = pa._views.pack(ts, pa._DTYPES, -1), pa._pack_views(ts, pa._DTYPES, -1)
    for t, a, b in zip(ts, with_ext[1], in_python[1]):
        assert (a is None and b is None) if t is None else bytes(pa.PaTensor.from_address(a)) == bytes(pa.PaTensor.from_address(b))
    for b in bad:
        assert pa._pack_views(b, pa._DTYPES, -1) == pa._views.pack(b, pa._DTYPES, -1)
    assert pa._pack_views((ts[0],), pa._DTYPES, 0) == 0  # on another device


def test_build_goes_on_without_the_views_extension(tmp_path, monkeypatch):
    """No C compiler or no Python headers: the library is built all the same, and is not built again for it."""
    spec = importlib.util.spec_from_file_location("_build_under_test", os.path.join(ROOT, "paged_kv_cache_385_b200", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "VIEWS", str(tmp_path / "_views.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "objects"))
    ran = []

    def run(cmd, **kw):
        if cmd[0] == "gcc":
            raise FileNotFoundError("gcc")
        ran.append(cmd)
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(b.subprocess, "run", run)
    with pytest.warns(UserWarning, match="_views"):
        assert b.build() == str(tmp_path / "lib.so")
    assert os.path.exists(tmp_path / "lib.so") and len(ran) == len(b.SOURCES) + 1
    with pytest.warns(UserWarning, match="_views"):
        b.build()
    assert len(ran) == len(b.SOURCES) + 1


def test_binding_names_the_tensor_that_is_missing(monkeypatch):
    """Packing and the check for absent tensors, with host tensors standing for device ones (no library call is made)."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    calls = ((pa.pa_rope_and_cache, rope_args, dict(zip(rope_args(), pa._ROPE_ARGS)), ("q", "q_out"), ()),
             (pa.pa_decode_tree, tree_args, dict(zip(tree_args(), pa._TREE_ARGS)), ("mask",), (5, 0.1, 2)),
             (pa.pa_commit_tree, commit_args, dict(zip(commit_args(), pa._COMMIT_ARGS)), ("new",), ()))
    for views in (pa._views, None):
        monkeypatch.setattr(pa, "_views", views)
        for call, make, names, optional, rest in calls:
            for key in make():
                if key in optional:
                    keep, refs_ = pa._views_of(list(names.values()), tuple(make(**{key: None}).values()),
                                               [names[k] for k in optional])
                    assert [r is None for r in refs_] == [k == key for k in make()]
                    continue
                with pytest.raises(ValueError, match=f"^{names[key]} is None$"):
                    call(*make(**{key: None}).values(), *rest)


class Elsewhere:
    """What the binding asks of a device tensor, for one that lies on a second GPU (or is empty, or has gaps)."""
    is_cuda, dtype = True, torch.int32

    def __init__(self, device=1, n=64, dense=True):
        self.device, self.n, self.dense = device, n, dense

    get_device = lambda self: self.device  # noqa: E731
    numel = lambda self: self.n  # noqa: E731
    element_size = lambda self: 4  # noqa: E731
    is_contiguous = lambda self: self.dense  # noqa: E731
    data_ptr = lambda self: 4096 if self.n else 0  # noqa: E731


@cpu_only
def test_words_and_workspaces_of_another_device_are_refused(monkeypatch):
    """A kernel that wrote them would fault; an empty error word would silently be the library's own."""
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # (host tensors stand for device ones)
    monkeypatch.setattr(pa, "_stream_handle", lambda stream: 0)
    rope_, tree_, commit_ = (lambda **kw: pa.pa_rope_and_cache(*rope_args().values(), **kw),
                             lambda **kw: pa.pa_decode_tree(*tree_args().values(), 5, 0.1, 2, **kw),
                             lambda **kw: pa.pa_commit_tree(*commit_args().values(), **kw))
    for call in (rope_, tree_, commit_):
        with pytest.raises(ValueError, match="error_word is on cuda:1, the current device is"):
            call(error_word=Elsewhere())
        with pytest.raises(ValueError, match="error_word is empty"):
            call(error_word=Elsewhere(-1, 0))
        with pytest.raises(pa.PagedAttentionError) as e:  # what is right gets as far as the device
            call(error_word=Elsewhere(-1))
        assert e.value.status == pa.PA_ERR_CUDA
    with pytest.raises(ValueError, match="workspace is on cuda:1, the current device is"):
        tree_(workspace=Elsewhere())
    with pytest.raises(ValueError, match="workspace must be contiguous"):
        tree_(workspace=Elsewhere(-1, dense=False))
    with pytest.raises(pa.PagedAttentionError) as e:
        tree_(workspace=Elsewhere(-1), error_word=Elsewhere(-1))
    assert e.value.status == pa.PA_ERR_CUDA


def test_angles_hold_their_bound():
    """The kernel's float64 turns, rounded to float32, against exact ones: 2^-22 of an angle up to 2^28 radians (3 * 2^-53
    of at most 2^25.4 turns and 2^-26 of a turn, times 2 pi: 2^-23.4 + 2^-23.3), and no such bound far beyond it."""
    pi = Fraction(int("314159265358979323846264338327950288419716939937510582097494459"), 10 ** 62)

    def worst(top, seed):
        r, most = random.Random(seed), 0.0
        for _ in range(3000):
            f = float(np.float32(r.uniform(0.01, 1.0)))
            pos = int(r.uniform(0.5, 1.0) * top / f)
            turns = np.float64(pos) * np.float64(f) * np.float64(0.15915494309189535)
            left = Fraction(float(np.float32(turns - np.rint(turns))))
            off = (Fraction(pos) * Fraction(f) / (2 * pi) - left) % 1
            most = max(most, 2 * math.pi * float(min(off, 1 - off)))
        return most

    assert worst(2.0 ** 28, 1) < 2.0 ** -22 and worst(1e6, 2) < 2.0 ** -23
    assert worst(2.0 ** 34, 3) > 2.0 ** -22
