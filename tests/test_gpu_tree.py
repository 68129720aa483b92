"""pa_decode_tree on the GPU against the float64 definition (oracle/tree.py)."""
import numpy as np
import pytest
import torch

import paged_kv_cache_385_b200 as pa
from tests.tree_case import TreeCase

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    pa.pa_read_device_error(clear=True)
    yield
    assert pa.pa_read_device_error(clear=True) == 0


def check(c: TreeCase, got: torch.Tensor):
    want, weight = c.oracle()
    n = c.start_host[-1]
    err = np.abs(got.double().cpu().numpy()[:n] - want[:n])
    over = err > c.bound(want, weight)[:n]
    assert not over.any(), (f"{int(over.sum())} of {over.size} values off, worst {np.nanmax(err):.3g} at "
                            f"{np.argwhere(over)[0].tolist()}")
    assert torch.all(got[n:] == 77.0)  # rows behind the last sequence


CASES = {
    # name: (kv, d, hkv, group, nodes per sequence, context per sequence, options)
    "one_token": ("f16", 64, 1, 1, [1], [1], {}),
    "one_token_128": ("bf16", 128, 2, 4, [1, 1], [1, 300], {}),
    "small": ("bf16", 128, 2, 4, [8], [100], {}),
    "whole_context_drafted": ("f16", 128, 1, 2, [16, 3, 64, 65], [16, 3, 64, 65], {}),
    "ragged": ("bf16", 128, 2, 4, [5, 0, 33, 1, 64], [5, 17, 1000, 63, 321], {}),
    "chain": ("f16", 128, 2, 4, [7, 64, 1], [500, 70, 65], {"masks": None}),
    "mha": ("f16", 128, 3, 1, [6, 17], [290, 48], {}),
    "group3": ("bf16", 128, 2, 3, [43, 9], [333, 31], {}),
    "group7_d64": ("f16", 64, 2, 7, [19, 37], [129, 400], {}),
    "group16": ("f16", 128, 1, 16, [8, 9], [256, 77], {}),
    "two_words": ("bf16", 128, 1, 2, [128, 100, 65], [200, 1100, 66], {}),
    "four_words": ("f16", 128, 1, 1, [256, 193], [1030, 193], {}),
    "four_words_chain": ("bf16", 64, 1, 5, [256], [300], {"masks": None}),
    "d64": ("bf16", 64, 4, 2, [13, 1, 50], [250, 16, 52], {}),
    "e4m3": ("e4m3", 128, 2, 8, [32, 7], [700, 65], {}),
    "e4m3_f16_query": ("e4m3", 128, 1, 4, [64, 5], [64, 2000], {"q": "f16"}),
    "e4m3_chain": ("e4m3", 128, 2, 3, [9, 1, 130], [1000, 1, 131], {"masks": None, "q": "f16"}),
    "capped": ("f16", 128, 2, 4, [12, 3], [400, 90], {"softcap": 2.0}),
    "capped_d64": ("bf16", 64, 2, 2, [12, 65], [400, 90], {"softcap": 30.0}),
    "capped_e4m3": ("e4m3", 128, 1, 8, [20], [300], {"softcap": 5.0}),
    "negative_scale": ("f16", 128, 1, 4, [9, 2], [150, 40], {"scale": -0.08}),
    "zero_scale": ("bf16", 128, 1, 4, [9], [150], {"scale": 0.0}),
    "zero_scale_few": ("f16", 128, 1, 2, [3], [150], {"scale": 0.0}),
    "tiny_cap": ("f16", 128, 1, 4, [9], [150], {"softcap": 1e-38}),
    "tiny_cap_few": ("bf16", 128, 1, 1, [9], [150], {"softcap": 1e-38, "scale": -1.0}),
    "long_split": ("bf16", 128, 1, 4, [10], [9001], {}),
    "long_split_e4m3": ("e4m3", 128, 1, 8, [3], [8000], {}),
    "long_split_d64": ("f16", 64, 2, 1, [5, 2], [7000, 33], {}),
    "few_rows": ("bf16", 128, 2, 4, [4, 1, 3, 0], [400, 1, 33, 9], {}),
    "few_rows_8": ("f16", 128, 3, 1, [8, 5, 1], [1200, 16, 17], {}),
    "few_rows_16": ("f16", 128, 2, 1, [16, 9, 15], [16, 1000, 47], {}),
    "few_rows_chain": ("bf16", 64, 2, 3, [5, 2], [500, 31], {"masks": None}),
    "few_rows_capped": ("f16", 128, 2, 2, [7, 8], [600, 64], {"softcap": 3.0}),
    "few_rows_d64": ("f16", 64, 4, 1, [3, 7], [100, 65], {}),
    "few_rows_e4m3": ("e4m3", 128, 2, 8, [2, 1], [900, 40], {}),
    "few_rows_e4m3_7": ("e4m3", 128, 1, 7, [1, 1, 1], [1, 320, 2000], {"q": "f16", "softcap": 10.0}),
    "few_rows_long": ("bf16", 128, 1, 8, [2], [20011], {}),
    "few_rows_long_e4m3": ("e4m3", 128, 2, 1, [7], [30000], {}),
    "few_rows_negative": ("f16", 128, 1, 2, [6], [150], {"scale": -0.1}),
    "few_rows_many": ("bf16", 64, 2, 2, [1, 3, 0, 2] * 60, [300, 3, 5, 70] * 60, {}),
    "many_short": ("f16", 64, 2, 2, [3, 1, 2, 5] * 40, [4, 1, 70, 33] * 40, {}),
}


@pytest.mark.parametrize("name", CASES)
def test_against_the_definition(name):
    kv, d, hkv, group, counts, lens, opts = CASES[name]
    c = TreeCase(kv, d, hkv, group, counts, lens, seed=len(name), extra_rows=3, **opts).to_device()
    check(c, c.run())


@pytest.mark.parametrize("n", [1, 15, 16, 17, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_tree_at_every_offset_of_a_tile(kv, n):
    """Contexts that end at, before and behind page and key-block borders, the tree straddling them."""
    lens = [n, n + 1, n + 15, n + 31, n + 48, n + 63, n + 64]
    c = TreeCase(kv, 128, 1, 2, [n] * len(lens), lens, seed=n).to_device()
    check(c, c.run())


def test_rows_that_see_nothing_are_zero():
    masks = [0, 0b10, 0, 0b1111]
    c = TreeCase("f16", 128, 1, 4, [4], [4], masks=masks, seed=3).to_device()
    got = c.run()
    check(c, got)
    assert torch.all(got[0] == 0) and torch.all(got[2] == 0)


def test_bits_behind_the_last_node_are_ignored():
    c = TreeCase("bf16", 128, 2, 2, [5, 70], [40, 170], seed=4).to_device()
    got = c.run().clone()
    full = torch.tensor(-1, dtype=torch.int64, device="cuda")
    for s, n in enumerate(c.counts):
        rows = c.mask[c.start_host[s]:c.start_host[s + 1]]
        for w in range(c.words):
            keep = max(0, min(64, n - 64 * w))
            if keep < 64:
                rows[:, w] |= full << keep
    assert torch.equal(c.run(out=torch.full_like(c.out, 77.0)), got)
    check(c, got)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("ctx", [12, 60, 1500])
@pytest.mark.parametrize("group", [1, 4])
def test_masked_rows_may_hold_anything(kv, ctx, group):
    """Keys and values of nodes that a node does not see are infinite or NaN: its row does not change."""
    c = TreeCase(kv, 128, 2, group, [12], [ctx], seed=5)
    before = c.to_device().run().clone()
    bad = 7  # the node that holds them: whoever sees it gives NaN, the others what they gave
    at = ctx - 12 + bad
    for pool, values in ((c.k_cache, (float("nan"), float("inf"))), (c.v_cache, (float("inf"), float("nan")))):
        row = pool[int(c.bt_host[0, at // 16]), :, at % 16]
        for h, v in enumerate(values):
            row[h] = torch.full((128,), v).to(pool.dtype).cuda()
    got = c.run(out=torch.full_like(c.out, 77.0))
    sees = torch.tensor([bool(m >> bad & 1) for m in c.masks])
    assert sees.any() and not sees.all()
    assert torch.equal(got[:12][~sees.cuda()], before[:12][~sees.cuda()])
    assert torch.isnan(got[:12][sees.cuda()]).all()


@pytest.mark.parametrize("group", [2, 4])
def test_infinite_values_reach_the_nodes_that_see_them(group):
    c = TreeCase("f16", 128, 1, group, [6], [300], seed=6).to_device()
    before = c.run().clone()
    at = 300 - 6 + 3
    c.v_cache[int(c.bt_host[0, at // 16]), 0, at % 16, 5] = float("inf")
    c.v_cache[int(c.bt_host[0, at // 16]), 0, at % 16, 6] = float("-inf")
    got = c.run()
    sees = torch.tensor([bool(m >> 3 & 1) for m in c.masks]).cuda()
    assert torch.all(got[:6][sees][..., 5] == float("inf")) and torch.all(got[:6][sees][..., 6] == float("-inf"))
    got[:6][..., 5:7] = before[:6][..., 5:7]
    assert torch.equal(got[:6][~sees], before[:6][~sees])
    rest = torch.ones(128, dtype=torch.bool)
    rest[5:7] = False
    assert torch.equal(got[:6][..., rest.cuda()], before[:6][..., rest.cuda()])


def test_single_nodes_agree_with_decode():
    """One drafted node per sequence is a decode step: both within their roundings of one exact row."""
    c = TreeCase("bf16", 128, 2, 4, [1] * 4, [1, 40, 700, 3000], seed=7).to_device()
    got = c.run()
    check(c, got)
    out = torch.empty_like(c.q)
    pa.pa_decode(out, c.q, c.k_cache, c.v_cache, c.bt, c.lens, c.scale, c.hkv, max_context_len=3000,
                 workspace=pa.decode_workspace(4, c.hq, c.hkv, 128, 3000))
    check(c, out)


def test_chain_agrees_with_prefill():
    c = TreeCase("f16", 128, 2, 4, [40, 7], [700, 90], masks=None, seed=8).to_device()
    check(c, c.run())
    out = torch.empty_like(c.q)
    pa.pa_prefill(out, c.q, c.k_cache, c.v_cache, c.bt, c.start, c.lens, 40, c.scale, c.hkv)
    check(c, out)


def test_strided_rows():
    c = TreeCase("bf16", 128, 2, 4, [9, 20], [100, 222], seed=9).to_device()
    T = c.q.shape[0]
    wide = torch.randn(T, c.hq + 4, 136, device="cuda").to(torch.bfloat16)
    q = wide[:, 2:2 + c.hq, 8:]
    q.copy_(c.q)
    out = torch.full((c.hq, T, 256), 77.0, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    c.run(out=out[..., :128], q=q)
    check(c, out[..., :128].contiguous())
    assert torch.all(out[..., 128:] == 77.0)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
@pytest.mark.parametrize("counts", [[9, 33, 1], [4, 1, 3]])
def test_placement_and_repetition_change_nothing(kv, counts):
    args = (kv, 128, 2, 4, counts, [100, 2222, 640])
    a = TreeCase(*args, seed=10).to_device()
    first = a.run().clone()
    for fill in (0, 0x7f):
        a.out.fill_(77.0)
        assert torch.equal(a.run(workspace=a.workspace(fill)), first)
    b = TreeCase(*args, seed=10, order=99).to_device()
    assert torch.equal(b.run(), first)


@pytest.mark.parametrize("counts", [[9, 40, 3], [2, 1, 4]])
def test_in_place(counts):
    """Contexts that are split and whole ones: every row's query is read before the row is written."""
    c = TreeCase("bf16", 128, 2, 4, counts, [9000, 90, 200], seed=16).to_device()
    want = c.run().clone()
    q = c.q.clone()
    c.run(out=q, q=q)
    T = sum(counts)
    assert torch.equal(q[:T], want[:T])


@pytest.mark.parametrize("kv,group", [("f16", 4), ("f16", 1), ("bf16", 4), ("e4m3", 8)])
def test_the_largest_cap(kv, group):
    """A capped score is off by at most 2^-20 of the cap: at 1024, 2^-10 on each weight and on their sum."""
    c = TreeCase(kv, 128, 2, group, [9, 7], [700, 64], seed=17, softcap=1024.0).to_device()
    got = c.run()
    want, weight = c.oracle()
    T = sum(c.counts)
    off = np.abs(got.double().cpu().numpy()[:T] - want[:T])
    assert np.all(off <= c.bound(want, weight)[:T] + 2 * 2.0 ** -10 * weight[:T])


def test_two_streams_at_once():
    """Calls that overlap on the GPU, each with its own workspace."""
    a = TreeCase("bf16", 128, 2, 4, [16, 5], [9000, 4000], seed=18).to_device()
    b = TreeCase("e4m3", 128, 2, 1, [7, 5, 3], [8000, 90, 2000], seed=19).to_device()
    runs = [(c, c.run().clone(), c.workspace(), torch.cuda.Stream(), torch.full_like(c.out, 77.0)) for c in (a, b)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, _, ws, stream, out in runs:
            c.run(out=out, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    for c, want, _, _, out in runs:
        assert torch.equal(out, want)


def test_default_context_bound_is_the_table():
    c = TreeCase("bf16", 128, 1, 4, [9], [100], seed=11).to_device()
    n = pa.pa_decode_tree_workspace_bytes(1, 4, 1, 128, 9, 16 * c.bt.shape[1])
    ws = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    check(c, c.run(max_context_len=0, workspace=ws))


def test_other_stream_and_graph():
    c = TreeCase("bf16", 128, 2, 4, [16, 5], [900, 4000], seed=12).to_device()
    want = c.run().clone()
    ws = c.workspace()
    side = torch.cuda.Stream()
    c.out.fill_(77.0)
    side.wait_stream(torch.cuda.current_stream())
    c.run(workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(c.out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        c.run(workspace=ws)
    # Lengths and values of a later step: the graph reads what the buffers hold then.
    d = TreeCase("bf16", 128, 2, 4, [5, 16], [77, 3000], seed=13).to_device()
    c.k_cache[:d.num_blocks].copy_(d.k_cache)
    c.v_cache[:d.num_blocks].copy_(d.v_cache)
    c.bt.fill_(-1)
    c.bt[:, :d.bt.shape[1]].copy_(d.bt)
    c.start.copy_(d.start), c.lens.copy_(d.lens), c.q.copy_(d.q), c.mask.copy_(d.mask)
    for _ in range(2):
        c.out.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        check(d, c.out)


@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
def test_many_runs_are_the_same(kv):
    """A race between the kernels' roles shows as bits that differ from run to run: ragged parts, rings that wrap."""
    for counts, lens in (([33, 64, 2, 17] * 4, [3000, 70, 999, 400] * 4), ([5, 9, 6], [60, 90, 200]), ([2, 4, 1] * 5, [4000, 40, 333] * 5)):
        c = TreeCase(kv, 128, 4, 4, counts, lens, seed=15).to_device()
        first = c.run().clone()
        for _ in range(40):
            assert torch.equal(c.run(out=torch.full_like(c.out, 77.0)), first)


@pytest.mark.parametrize("kv", ["f16", "e4m3"])
@pytest.mark.parametrize("group", [1, 4])
def test_out_of_contract_sequences_are_left_alone(kv, group):
    """A sequence the device finds out of contract sets its bit; the others are computed."""
    c = TreeCase(kv, 128, 2, group, [5, 9, 6], [60, 90, 200], seed=14).to_device()
    want, weight = c.oracle()
    bound = c.bound(want, weight)
    word = torch.zeros(1, dtype=torch.int32, device="cuda")

    def right(got, a, b):  # (where contexts are cut goes by the whole batch's lengths, so bits may differ)
        return bool((np.abs(got[a:b].double().cpu().numpy() - want[a:b]) <= bound[a:b]).all())

    def rerun(**kw):
        word.zero_()
        return c.run(out=torch.full_like(c.out, 77.0), error_word=word, **kw)

    lens = c.lens.clone()
    for bad in (4, 0, -3, 16 * c.bt.shape[1] + 1, 2 ** 31 - 1):  # shorter than its nodes, or past the table
        c.lens[0] = bad
        got = rerun()
        assert int(word) == pa.PA_DEVERR_CTX_RANGE, bad
        assert torch.all(got[:5] == 77.0) and right(got, 5, 20)
        c.lens.copy_(lens)
    got = rerun(max_context_len=150)
    assert int(word) == pa.PA_DEVERR_CTX_RANGE and torch.all(got[14:20] == 77.0) and right(got, 0, 14)
    start = c.start.clone()
    for at, value in ((3, 10 ** 6), (0, -1), (3, 13)):  # rows outside q; a negative count
        c.start[at] = value
        rerun()
        assert int(word) == pa.PA_DEVERR_CTX_RANGE, (at, value)
        c.start.copy_(start)
    c.bt[1, 2] = c.num_blocks
    got = rerun()
    assert int(word) == pa.PA_DEVERR_BAD_BLOCK
    assert right(got, 0, 5) and right(got, 14, 20)
    assert pa.pa_read_device_error(clear=True) == 0


# ---- non-finite rows, empty masks and signs in every form ------------------------------------------------
# Nodes and group reach the warp-level form (up to 16 rows), one tile (up to 128) and two (above).

FORMS = {"warp": (4, 4), "one_tile": (33, 3), "one_tile_words": (100, 1), "two_tiles": (40, 4), "two_tiles_words": (200, 1),
         "two_items": (72, 16)}


def poison(c, pool, node, rows):
    """Row `rows[h]` of KV head h in the place of sequence 0's node."""
    at = c.lens_host[0] - c.counts[0] + node
    for h, row in enumerate(rows):
        pool[int(c.bt_host[0, at // 16]), h, at % 16] = row.to(pool.dtype).cuda()


@pytest.mark.parametrize("before", [0, 5, 2000])
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv,cap", [("f16", 0.0), ("bf16", 0.0), ("e4m3", 0.0), ("bf16", 20.0), ("e4m3", 20.0)])
def test_masked_rows_may_hold_anything_in_every_form(kv, cap, form, before):
    """Several nodes of one tree, in every word of the masks, hold NaN and infinities."""
    n, group = FORMS[form]
    c = TreeCase(kv, 128, 2, group, [n, 3], [n + before, 40], seed=21, softcap=cap, extra_rows=2).to_device()
    want = c.run().clone()
    bad = [b for b in (3, 33, 70, 130, 190) if b < n]
    full = [torch.full((128,), x) for x in (float("nan"), float("inf"))]
    for i, b in enumerate(bad):
        poison(c, c.k_cache, b, full if i % 2 else full[::-1])
        poison(c, c.v_cache, b, full[::-1] if i % 2 else full)
    got = c.run(out=torch.full_like(c.out, 77.0))
    sees = torch.tensor([any(m >> b & 1 for b in bad) for m in c.masks[:n]] + [False] * 5).cuda()
    assert sees.any() and not sees[:n].all()
    assert torch.equal(got[~sees], want[~sees])
    assert torch.isnan(got[sees]).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv", ["f16", "bf16", "e4m3"])
def test_values_of_seen_nodes_reach_their_column(kv, form):
    """Single non-finite elements of drafted V rows, in a context that is cut into parts."""
    n, group = FORMS[form]
    c = TreeCase(kv, 128, 2, group, [n], [n + 3000], seed=22).to_device()
    before = c.run().clone()
    odd = [float("nan")] * 3 if kv == "e4m3" else [float("inf"), float("-inf"), float("nan")]
    nodes = [b for b in (1, 33, 70, 130, 190) if b < n]
    for i, b in enumerate(nodes):
        at = 3000 + b
        c.v_cache[int(c.bt_host[0, at // 16]), :, at % 16, 7 + 20 * i] = torch.tensor(odd[i % 3]).to(c.v_cache.dtype).cuda()
    got = c.run(out=torch.full_like(c.out, 77.0))
    for i, b in enumerate(nodes):
        sees = torch.tensor([bool(m >> b & 1) for m in c.masks]).cuda()
        column = got[sees][..., 7 + 20 * i].float()
        want = torch.full_like(column, odd[i % 3])
        assert torch.equal(column.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0)), b
        got[sees, :, 7 + 20 * i] = before[sees, :, 7 + 20 * i]
    assert torch.equal(got, before)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv,cap", [("f16", 0.0), ("bf16", 20.0), ("e4m3", 0.0), ("e4m3", 20.0)])
def test_rows_that_see_nothing_are_zero_in_every_form(kv, cap, form):
    n, group = FORMS[form]
    masks = [0 if i % 3 == 0 else (1 << i if i % 3 == 1 else 1 << (i // 2)) for i in range(n)]
    c = TreeCase(kv, 128, 2, group, [n], [n], masks=masks, softcap=cap, seed=23, extra_rows=1).to_device()
    got = c.run()
    check(c, got)
    assert torch.all(got[:n:3] == 0)
    c.masks = [0] * n
    c.mask.zero_()
    got = c.run(out=torch.full_like(c.out, 77.0))
    assert torch.all(got[:n] == 0) and torch.all(got[n:] == 77.0)


@pytest.mark.parametrize("before", [0, 2000])
@pytest.mark.parametrize("form", FORMS)
def test_rows_whose_scores_are_all_minus_infinity_are_zero(form, before):
    n, group = FORMS[form]
    c = TreeCase("bf16", 128, 2, group, [n], [n + before], seed=24).to_device()
    c.q[..., 0] = c.q[..., 0].abs() + 1
    c.k_cache[..., 0] = float("-inf")
    assert torch.all(c.run() == 0)


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv,cap", [("f16", 0.0), ("bf16", 20.0)])
def test_a_scale_of_zero_makes_infinite_products_nan(kv, cap, form):
    """0 times an infinite product is NaN, for the rows that see its key; the others weigh all that they see alike."""
    n, group = FORMS[form]
    c = TreeCase(kv, 128, 2, group, [n], [n + 700], seed=25, scale=0.0, softcap=cap).to_device()
    want = c.run().clone()
    check(c, want)
    spike = torch.zeros(128)
    spike[5] = float("inf")
    c.q[..., 5] = 1.0
    poison(c, c.k_cache, 2, [spike, spike])
    got = c.run(out=torch.full_like(c.out, 77.0))
    sees = torch.tensor([bool(m >> 2 & 1) for m in c.masks]).cuda()
    assert torch.isnan(got[sees]).all()
    assert torch.equal(got[~sees], want[~sees])
    at = 100  # a token of the context, which every node sees
    c.k_cache[int(c.bt_host[0, at // 16]), :, at % 16] = spike.to(c.k_cache.dtype).cuda()
    assert torch.isnan(c.run()).all()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv,q,cap", [("e4m3", "bf16", 0.0), ("e4m3", "f16", 0.0), ("e4m3", "bf16", 4.0), ("bf16", "", 0.0)])
def test_negative_scales_in_every_form(kv, q, cap, form):
    n, group = FORMS[form]
    c = TreeCase(kv, 128, 1, group, [n, 2], [n + 150, 40], seed=26, scale=-0.09, q=q, softcap=cap, extra_rows=1).to_device()
    check(c, c.run())


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("kv,d", [("f16", 128), ("bf16", 64), ("e4m3", 128)])
def test_caps_in_every_form(kv, d, form):
    n, group = FORMS[form]
    c = TreeCase(kv, d, 1, group, [n, 1], [n + 333, 1], seed=27, softcap=3.0, extra_rows=1).to_device()
    check(c, c.run())


def test_calls_without_the_views_extension(monkeypatch):
    c = TreeCase("bf16", 128, 2, 4, [9, 2], [150, 40], seed=28).to_device()
    want = c.run().clone()
    monkeypatch.setattr(pa, "_views", None)
    assert torch.equal(c.run(out=torch.full_like(c.out, 77.0)), want)
    c.mask = None
    c.masks = None
    check(c, c.run(out=torch.full_like(c.out, 77.0)))


def replay_us(call):
    """Microseconds of a call, from the fastest of some replays of a graph of 20."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(20):
            call()
    best = float("inf")
    for _ in range(10):
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        graph.replay()
        end.record()
        torch.cuda.synchronize()
        best = min(best, begin.elapsed_time(end) * 50)
    return best


@pytest.mark.parametrize("n", [4, 16, 64])
def test_slots_without_nodes(n):
    """A padded batch: hundreds of empty slots before, between and behind the sequences change no row, and cost no
    multiple of the batch's time (one load's latency each was eight times it)."""
    real, lens = [n, 1, n], [700, 300, 33 + n]
    c = TreeCase("bf16", 128, 2, 4, real, lens, masks=None, seed=29).to_device()
    ws = c.workspace()
    plain = replay_us(lambda: c.run(workspace=ws))
    table = c.bt
    for gap in (1, 7, 8, 9, 600):
        for before, between, behind in ((gap, 0, 0), (0, gap, 0), (0, 0, gap), (gap, gap, gap)):
            slots = [before, before + 1 + between, before + 2 + 2 * between]
            B = slots[-1] + 1 + behind
            c.bt = torch.full((B, table.shape[1]), -1, dtype=torch.int32, device="cuda")
            counts, ctx = [0] * B, [0] * B
            for i, s in enumerate(slots):
                c.bt[s] = table[i]
                counts[s], ctx[s] = real[i], lens[i]
            c.start = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
            c.lens = torch.tensor(ctx, dtype=torch.int32, device="cuda")
            m = pa.pa_decode_tree_workspace_bytes(B, c.hq, c.hkv, 128, n, max(lens))
            ws = torch.empty(m, dtype=torch.uint8, device="cuda")
            check(c, c.run(out=torch.full_like(c.out, 77.0), workspace=ws))
            if gap == 600:
                took = replay_us(lambda: c.run(workspace=ws))
                assert took < 2 * plain + 5, (before, between, behind, plain, took)


@pytest.mark.parametrize("counts", [[9, 3], [2, 4]])
def test_rows_before_the_first_sequence(counts):
    """query_start may begin behind some rows: they are neither read nor written."""
    c = TreeCase("bf16", 128, 2, 4, counts, [150, 40], seed=30).to_device()
    want = c.run().clone()
    q = torch.cat([torch.full_like(c.q[:5], float("nan")), c.q])
    c.mask = torch.cat([torch.full_like(c.mask[:1].expand(5, -1), -1), c.mask])
    c.start += 5
    got = c.run(out=torch.full_like(q, 77.0), q=q)
    assert torch.equal(got[5:], want) and torch.all(got[:5] == 77.0)
