"""pa_commit_tree on the GPU, bit for bit against the oracle; and a whole step of drafted tokens."""
import random

import numpy as np
import pytest
import torch

import paged_kv_cache_385_b200 as pa
from oracle import attention, tree
from tests.tree_case import TreeCase, mask_words

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error():
    pa.pa_read_device_error(clear=True)
    yield
    assert pa.pa_read_device_error(clear=True) == 0


def commit(c, paths, width=None, **kw):
    width = width or max([1] + [len(p) for p in paths])
    acc = torch.full((len(paths), width), -7, dtype=torch.int32)
    for s, p in enumerate(paths):
        acc[s, :len(p)] = torch.tensor(p, dtype=torch.int32)
    new = torch.full((len(paths),), -1, dtype=torch.int32, device="cuda")
    pa.pa_commit_tree(c.k_cache, c.v_cache, c.bt, c.start, c.lens, acc.cuda(),
                      torch.tensor([len(p) for p in paths], dtype=torch.int32, device="cuda"), new, **kw)
    return new


def check(c, paths, new):
    k, v, lens = tree.commit(c.host_pool(0), c.host_pool(1), c.bt_host.numpy(), c.start_host, c.lens_host, paths)
    assert new.tolist() == lens
    for got, want in ((c.k_cache, k), (c.v_cache, v)):
        assert np.array_equal(got.view(torch.uint8).reshape(want.shape).cpu().numpy(), want)


@pytest.mark.parametrize("kv,d", [("f16", 64), ("bf16", 128), ("e4m3", 128), ("e4m3", 64), ("f16", 8)])
def test_paths(kv, d):
    paths = [[0, 2, 3, 11], [], [0], list(range(1, 40)), [3, 4, 5], [0, 1, 2], [39], list(range(0, 40, 3))]
    c = TreeCase(kv, d, 3, 1, [40] * 8, [40, 41, 55, 100, 64, 48, 300, 40], seed=1).to_device()
    check(c, paths, commit(c, paths, width=41))


def test_long_paths_and_ragged_trees():
    r = random.Random(2)
    counts = [256, 1, 0, 200, 17, 64]
    paths = [sorted(r.sample(range(n), r.randint(0, n))) for n in counts]
    paths[0] = list(range(1, 256))
    c = TreeCase("bf16", 128, 2, 1, counts, [256 + 3, 1, 20, 1000, 33, 70], seed=3).to_device()
    check(c, paths, commit(c, paths))


def test_bad_paths_move_nothing():
    counts, lens = [6] * 8, [20] * 8
    c = TreeCase("f16", 64, 2, 1, counts, lens, seed=4).to_device()
    good = [0, 3, 5]
    paths = [[1, 0], good, [2, 2], [0, 6], [-1, 2], [0, 1, 2, 3, 4, 5, 5], good, good]
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = commit(c, paths, error_word=word)
    assert int(word) == pa.PA_DEVERR_TREE
    moved = [p if i in (1, 6, 7) else [0, 1, 2, 3, 4, 5] for i, p in enumerate(paths)]
    check(c, moved, new)  # what is refused keeps its rows and its length (as an identical path would)
    assert new.tolist() == [17 if i in (1, 6, 7) else 20 for i in range(8)]


def test_lengths_out_of_range():
    c = TreeCase("f16", 64, 1, 1, [6, 6, 6], [20, 30, 40], seed=5).to_device()
    c.lens[0], c.lens[2] = 5, 16 * c.bt.shape[1] + 1
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = commit(c, [[0, 2], [1, 5], [1]], error_word=word)
    assert int(word) == pa.PA_DEVERR_CTX_RANGE
    assert new.tolist() == [5, 26, 16 * c.bt.shape[1] + 1]
    k, v, _ = tree.commit(c.host_pool(0), c.host_pool(1), c.bt_host.numpy(), c.start_host, c.lens_host, [[], [1, 5], []])
    assert np.array_equal(c.k_cache.view(torch.uint8).reshape(k.shape).cpu().numpy(), k)
    assert np.array_equal(c.v_cache.view(torch.uint8).reshape(v.shape).cpu().numpy(), v)


def test_bad_block_skips_the_row():
    c = TreeCase("f16", 64, 1, 1, [20], [40], seed=6).to_device()
    c.bt[0, 2] = c.num_blocks  # positions 32 .. 47: nodes 12 ..
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    commit(c, [[1, 3, 13]], error_word=word)
    assert int(word) == pa.PA_DEVERR_BAD_BLOCK
    k, _, _ = tree.commit(c.host_pool(0), c.host_pool(1), c.bt_host.numpy(), c.start_host, c.lens_host, [[1, 3]])
    assert np.array_equal(c.k_cache.view(torch.uint8).reshape(k.shape).cpu().numpy(), k)


def test_without_new_lengths_on_a_stream():
    c = TreeCase("bf16", 128, 2, 1, [8, 8], [50, 8], seed=7).to_device()
    acc = torch.tensor([[0, 4], [2, 3]], dtype=torch.int32, device="cuda")
    taken = torch.full((2,), 2, dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    pa.pa_commit_tree(c.k_cache, c.v_cache, c.bt, c.start, c.lens, acc, taken, stream=side)
    side.synchronize()
    check(c, [[0, 4], [2, 3]], torch.tensor([44, 2]))


@pytest.mark.parametrize("kv", ["bf16", "e4m3"])
def test_a_step_of_drafted_tokens(kv):
    """Write a tree's keys and values, attend, commit its accepted path, and decode the next token: the
    cache and the outputs are those of the accepted tokens written one after another."""
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[kv]
    B, hkv, group, d, words = 3, 2, 4, 128, 1
    hq, scale, ks, vs = hkv * group, 128 ** -0.5, 0.02, 0.02
    if kv != "e4m3":
        ks = vs = 1.0
    g = torch.Generator().manual_seed(8)
    history, nodes = [37, 5, 160], [13, 6, 9]
    parents = [[-1] + [(i - 1) // 2 for i in range(1, n)] for n in nodes]
    accepted = [[0, 2, 5, 12], [0], [0, 1, 4]]
    alloc = pa.BlockAllocator(64, torch.randperm(64, generator=g).tolist())
    bt_host = pa.build_block_tables(alloc, [h + n for h, n in zip(history, nodes)], 16)
    bt = bt_host.cuda()
    kc, vc = (torch.zeros(64, hkv, 16, d, device="cuda").to(dt) for _ in range(2))
    inv = pa.pa_rope_inv_freq(d, 10000.0).cuda()

    def rows(n, h):
        return torch.randn(n, h, d, generator=g).to(torch.bfloat16)

    def write(k_pool, v_pool, seqs, places, positions, key, value, q=None):
        out = None if q is None else torch.empty_like(q.cuda())
        pa.pa_rope_and_cache(out, None if q is None else q.cuda(), key.cuda(), value.cuda(),
                             torch.tensor(positions).cuda(), inv, pa.pa_slots_for_positions(bt_host, seqs, places).cuda(),
                             k_pool, v_pool, k_scale=ks, v_scale=vs)
        return out

    hist = [(rows(h, hkv), rows(h, hkv)) for h in history]
    draft = [(rows(n, hkv), rows(n, hkv)) for n in nodes]
    q = rows(sum(nodes), hq)
    masks, depth, seqs, places, positions = [], [], [], [], []
    for s, n in enumerate(nodes):
        write(kc, vc, [s] * history[s], list(range(history[s])), list(range(history[s])), *hist[s])
        seen, deep = [], []
        for i, p in enumerate(parents[s]):
            seen.append((seen[p] if p >= 0 else 0) | 1 << i)
            deep.append(deep[p] + 1 if p >= 0 else 0)
        masks += seen
        depth.append(deep)
        seqs += [s] * n
        places += [history[s] + i for i in range(n)]
        positions += [history[s] + x for x in deep]
    plain = [kc.clone(), vc.clone()]
    q_rot = write(kc, vc, seqs, places, positions, torch.cat([k for k, _ in draft]), torch.cat([v for _, v in draft]), q)
    start = torch.tensor([0, 13, 19, 28], dtype=torch.int32, device="cuda")
    lens = torch.tensor([h + n for h, n in zip(history, nodes)], dtype=torch.int32, device="cuda")
    out = torch.empty_like(q_rot)
    ws = torch.empty(pa.pa_decode_tree_workspace_bytes(B, hq, hkv, d, 13, 256), dtype=torch.uint8, device="cuda")
    pa.pa_decode_tree(out, q_rot, kc, vc, bt, start, lens, mask_words(masks, words).cuda(), 13, scale, hkv, k_scale=ks,
                      v_scale=vs, max_context_len=256, workspace=ws if ws.numel() else None)
    acc = torch.full((B, 4), -1, dtype=torch.int32)
    for s, p in enumerate(accepted):
        acc[s, :len(p)] = torch.tensor(p)
    new = torch.empty_like(lens)
    pa.pa_commit_tree(kc, vc, bt, start, lens, acc.cuda(), torch.tensor([4, 1, 3], dtype=torch.int32).cuda(), new)
    assert new.tolist() == [h + len(p) for h, p in zip(history, accepted)]

    # The same tokens without a tree: written one by one, each position decoded as it comes.
    for s, path in enumerate(accepted):
        k, v = draft[s]
        write(*plain, [s] * len(path), [history[s] + i for i in range(len(path))],
              [history[s] + i for i in range(len(path))], k[path], v[path])
    for s, n in enumerate(new.tolist()):
        t = torch.arange(n)
        at = (bt_host[s, t // 16].long().cuda(), slice(None), (t % 16).cuda())
        for a, b in zip((kc, vc), plain):
            assert torch.equal(a.view(torch.uint8)[at], b.view(torch.uint8)[at])
    byte_pools = [p.view(torch.uint8).reshape(64, hkv, 16, -1).cpu().numpy() for p in plain]
    for s, path in enumerate(accepted):
        for i, node in enumerate(path):
            row = int(start[s]) + node
            want = attention.decode_paged(q_rot[row:row + 1].double().cpu().numpy(), *byte_pools, bt_host[s:s + 1].numpy(),
                                          [history[s] + i + 1], scale, hkv, kv, ks, vs)
            assert np.abs(out[row].double().cpu().numpy() - want[0]).max() < (3e-2 if kv == "e4m3" else 1.5e-2)
    nxt = rows(B, hq).cuda()
    outs = [torch.empty_like(nxt) for _ in range(2)]
    for o, pools in zip(outs, ((kc, vc), plain)):
        pa.pa_decode(o, nxt, *pools, bt, new, scale, hkv, k_scale=ks, v_scale=vs, max_context_len=256)
    assert torch.equal(*outs)


@pytest.mark.parametrize("kv,group", [("bf16", 4), ("e4m3", 4), ("bf16", 1)])
def test_the_far_end_of_a_large_pool(kv, group):
    """A pool of more than 2^32 elements, its last blocks in use: every call gives what it gives in a small one."""
    c = TreeCase(kv, 128, 8, group, [9, 40], [150, 400], seed=9).to_device()
    want = c.run().clone()
    raw = torch.uint8 if kv == "e4m3" else torch.int16
    blocks = (1 << 32) // (8 * 16 * 128) + 1000
    off = blocks - c.num_blocks
    small, far = [c.k_cache, c.v_cache], []
    for p in small:
        far.append(torch.zeros(blocks, 8, 16, 128, dtype=p.dtype, device="cuda"))
        far[-1].view(raw)[off:] = p.view(raw)
    far_bt = torch.where(c.bt >= 0, c.bt + off, c.bt)
    g = torch.Generator().manual_seed(10)
    key, value = (torch.randn(7, 8, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slots, positions = torch.arange(7, device="cuda") * 13 + 5, torch.arange(7, device="cuda") * 1000
    inv = pa.pa_rope_inv_freq(128).cuda()
    accepted = torch.tensor([[0, 3, 7], [1, 20, 39]], dtype=torch.int32, device="cuda")
    taken = torch.full((2,), 3, dtype=torch.int32, device="cuda")
    out, bt = torch.full_like(c.out, 77.0), c.bt
    c.k_cache, c.v_cache, c.bt = *far, far_bt
    assert torch.equal(c.run(out=out), want)
    for pools, table, first in ((small, bt, 0), (far, far_bt, 16 * off)):
        pa.pa_commit_tree(*pools, table, c.start, c.lens, accepted, taken)
        pa.pa_rope_and_cache(None, None, key, value, positions, inv, slots + first, *pools, k_scale=0.02, v_scale=0.02)
    for a, b in zip(far, small):
        assert torch.equal(a.view(raw)[off:], b.view(raw)) and not a.view(raw)[:off].any()


@pytest.mark.parametrize("group,nodes", [(4, [13, 6, 9]), (1, [3, 5, 2])])
def test_a_captured_step(group, nodes):
    """Write, attend and commit captured into one graph: every replay gives what the calls one by one give."""
    hkv, history = 2, [370, 5, 160]
    c = TreeCase("bf16", 128, hkv, group, nodes, [h + n for h, n in zip(history, nodes)], seed=11).to_device()
    T, slots = sum(nodes), []
    for s, (h, n) in enumerate(zip(history, nodes)):
        slots += pa.pa_slots_for_positions(c.bt_host, [s] * n, list(range(h, h + n))).tolist()
    slots = torch.tensor(slots, device="cuda")
    positions = torch.arange(T, device="cuda") % 7 + 100
    inv = pa.pa_rope_inv_freq(128).cuda()
    accepted = torch.tensor([[0, 2], [0, 3], [1, -1]], dtype=torch.int32, device="cuda")
    taken = torch.tensor([2, 2, 1], dtype=torch.int32, device="cuda")
    key, value, q = (torch.empty(T, h, 128, dtype=torch.bfloat16, device="cuda") for h in (hkv, hkv, hkv * group))
    q_out, new, ws = torch.empty_like(q), torch.empty_like(c.lens), c.workspace()

    def step():
        pa.pa_rope_and_cache(q_out, q, key, value, positions, inv, slots, c.k_cache, c.v_cache)
        c.run(q=q_out, workspace=ws)
        pa.pa_commit_tree(c.k_cache, c.v_cache, c.bt, c.start, c.lens, accepted, taken, new)

    def state():
        return [t.view(torch.int16).clone() for t in (q_out, c.out, c.k_cache, c.v_cache)] + [new.clone()]

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for t in (key, value, q):
        t.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (1, 2, 3):
        g = torch.Generator().manual_seed(seed)
        fresh = [torch.randn(t.shape, generator=g).to(torch.bfloat16).cuda() for t in (key, value, q)]
        pools = c.k_cache.clone(), c.v_cache.clone()
        got = []
        for run in (graph.replay, step):
            for t, x in zip((key, value, q, c.k_cache, c.v_cache), (*fresh, *pools)):
                t.copy_(x)
            c.out.fill_(77.0), q_out.fill_(77.0), new.fill_(-1)
            run()
            torch.cuda.synchronize()
            got.append(state())
        assert all(torch.equal(a, b) for a, b in zip(*got))
