"""The speculative-decoding operators over the paged cache, as cases to be measured.

A serving step that verifies drafted tokens runs three operators next to this library's decode and
prefill. All of them work on the same pool, block tables and lengths:

* ``rope``: ``pa_rope_and_cache`` rotates the queries and keys of new tokens by their positions and
  writes keys and values into their slots (16-bit or e4m3 pages);
* ``tree``: ``pa_decode_tree`` lets each drafted node attend over its sequence's whole context and
  over the drafted nodes that its mask names;
* ``commit``: ``pa_commit_tree`` moves the accepted nodes' rows to the front of the drafted region
  and gives the new lengths.

A case's lengths come from its own ``lens_seed``, so ``work`` knows them; the values, the pages'
places and the trees come from the seed given to ``prepare``.
"""
import math
import random

import torch

own = False

_KV = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
_Q = {"f16": torch.float16, "bf16": torch.bfloat16}
_ELEM = {"f16": 2, "bf16": 2, "e4m3": 1}
_PAGE = 16


def listed():
    return [
        # One conversation, a small tree: what a single user waits for at each step.
        _tree("tree_one_user", seqs=1, hq=32, hkv=8, d=128, kv="bf16", lo=777, hi=777, nlo=8, nhi=8),
        # The 8B-shaped batch of the decode benchmark, 16 drafted nodes each, ragged contexts.
        _tree("tree_8b_batch", seqs=64, hq=32, hkv=8, d=128, kv="bf16", lo=128, hi=8192, nlo=16, nhi=16),
        # Short drafted chains, one query head per KV head (the 7B-shaped batch), capped scores.
        _tree("tree_7b_mha_capped", seqs=32, hq=32, hkv=32, d=128, kv="f16", lo=2048, hi=2048, nlo=5, nhi=7, cap=30.0,
              chain=True),
        # Wide trees over few sequences: up to 200 nodes, the ragged ones in between.
        _tree("tree_wide", seqs=4, hq=32, hkv=8, d=128, kv="bf16", lo=1000, hi=9001, nlo=150, nhi=200),
        # The 70B-shaped long-context batch with 8-bit pages: the largest work.
        _tree("tree_70b_e4m3", seqs=8, hq=64, hkv=8, d=128, kv="e4m3", lo=32768, hi=131072, nlo=32, nhi=32),
        # Small heads, odd lengths and node counts.
        _tree("tree_d64", seqs=9, hq=12, hkv=4, d=64, kv="f16", lo=1, hi=1901, nlo=1, nhi=13),
        # One decode step of the 8B-shaped batch: latency.
        _rope("rope_step", tokens=64, hq=32, hkv=8, d=128, rot=128, kv="bf16", q="bf16", far=8192),
        # A prompt's prefill.
        _rope("rope_prefill", tokens=16384, hq=32, hkv=8, d=128, rot=128, kv="bf16", q="bf16", far=131072),
        # Interleaved pairs over half of the head, 8-bit pages, an odd token count, far positions.
        _rope("rope_e4m3_part", tokens=4097, hq=64, hkv=8, d=128, rot=64, kv="e4m3", q="bf16", far=1000000, pairs=True),
        # A few sequences accept a few nodes each: latency.
        _commit("commit_few", seqs=4, hkv=8, d=128, kv="bf16", lo=100, hi=900, nodes=16, path=4),
        # The 8B-shaped batch.
        _commit("commit_batch", seqs=64, hkv=8, d=128, kv="bf16", lo=128, hi=2048, nodes=64, path=9),
        # Long accepted paths of many sequences, 8-bit pages.
        _commit("commit_long_e4m3", seqs=500, hkv=8, d=128, kv="e4m3", lo=150, hi=600, nodes=130, path=60),
    ]


def _tree(name, seqs, hq, hkv, d, kv, lo, hi, nlo, nhi, cap=0.0, chain=False, lens_seed=1):
    return {"name": name, "op": "tree", "seqs": seqs, "hq": hq, "hkv": hkv, "d": d, "kv": kv, "lo": lo, "hi": hi,
            "nlo": nlo, "nhi": nhi, "cap": cap, "chain": chain, "lens_seed": lens_seed}


def _rope(name, tokens, hq, hkv, d, rot, kv, q, far, pairs=False):
    return {"name": name, "op": "rope", "tokens": tokens, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "kv": kv, "q": q,
            "far": far, "pairs": pairs}


def _commit(name, seqs, hkv, d, kv, lo, hi, nodes, path, lens_seed=1):
    return {"name": name, "op": "commit", "seqs": seqs, "hkv": hkv, "d": d, "kv": kv, "lo": lo, "hi": hi,
            "nodes": nodes, "path": path, "lens_seed": lens_seed}


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("tree", "tree", "rope", "commit"))
    kv = rng.choice(("f16", "bf16", "e4m3"))
    d = 128 if kv == "e4m3" else rng.choice((64, 128, 128))
    if op == "tree":
        group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16))
        hkv = _log(rng, 1, 32)
        hkv = max(1, min(hkv, 128 // group))
        seqs, nhi, hi = _log(rng, 1, 64), _log(rng, 1, 256), _log(rng, 1, 131072)
        # No more context rows, and no more scores, than the largest listed case has at its longest.
        hi = min(hi, (500 << 20) // (seqs * hkv * d * _ELEM[kv]), (1 << 30) // (seqs * hkv * group * nhi))
        hi = max(hi, nhi)
        lo = rng.randint(1, hi)
        c = _tree("", seqs, group * hkv, hkv, d, kv, lo, hi, rng.randint(1, nhi), nhi, rng.choice((0.0, 0.0, 50.0)),
                  rng.random() < 0.3, rng.randrange(1 << 20))
    elif op == "rope":
        hkv = _log(rng, 1, 16)
        rot = rng.choice((d, d, d // 2, 24))
        c = _rope("", _log(rng, 1, 16384), hkv * rng.choice((1, 3, 4)), hkv, d, rot, kv,
                  kv if kv != "e4m3" else rng.choice(("f16", "bf16")), _log(rng, 1024, 1000000), rng.random() < 0.4)
    else:
        nodes = _log(rng, 2, 200)
        lo = nodes + rng.randint(0, 200)
        c = _commit("", _log(rng, 1, 500), rng.choice((1, 2, 4, 8)), d, kv, lo, lo + rng.randint(0, 300), nodes,
                    rng.randint(1, max(1, min(nodes // 2, 60))), rng.randrange(1 << 20))
    del c["name"]
    return c


def _lens(case):
    """(context lengths, drafted nodes) of a case's sequences, or (lengths, accepted) for a commit."""
    r = random.Random(case["lens_seed"])
    if case["op"] == "commit":
        return ([r.randint(case["lo"], case["hi"]) for _ in range(case["seqs"])],
                [r.randint(1, case["path"]) for _ in range(case["seqs"])])
    nodes = [r.randint(case["nlo"], case["nhi"]) for _ in range(case["seqs"])]
    return [max(n, r.randint(case["lo"], case["hi"])) for n in nodes], nodes


def work(case):
    c, e = case, _ELEM[case["kv"]]
    if c["op"] == "rope":
        q, kv = c["tokens"] * c["hq"] * c["d"], c["tokens"] * c["hkv"] * c["d"]
        return {"bytes": 4 * q + 2 * kv * (2 + e) + 16 * c["tokens"], "flops": 3 * (q + kv)}
    lens, counts = _lens(c)
    if c["op"] == "commit":
        moved = sum(max(0, a - _kept(a)) for a in counts)
        return {"bytes": 4 * moved * c["hkv"] * c["d"] * e + 4 * sum(counts) + 16 * c["seqs"], "flops": 0}
    rows = sum(counts)
    return {"bytes": 2 * sum(lens) * c["hkv"] * c["d"] * e + 4 * rows * c["hq"] * c["d"],
            "flops": 4 * c["hq"] * c["d"] * sum(n * (k - n) + n for k, n in zip(lens, counts))}


def _kept(accepted):
    """The leading nodes of an accepted path that already lie where they belong (the root, and some more)."""
    return (accepted + 2) // 3


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, dtype):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(g, blocks, case):
    """A cache of random rows; for e4m3, codes of normal values at the scale that the case uses."""
    x = torch.randn(blocks, case["hkv"], _PAGE, case["d"], generator=g, device="cuda")
    return x.div_(_scale(case)).to(_KV[case["kv"]])


def _scale(case):
    return 1.0 / 64 if case["kv"] == "e4m3" else 1.0


def _tables(g, lens):
    """Block tables of scattered pages: [seqs, widest] int32 (-1 behind each row's last), and the pool's blocks."""
    need = torch.tensor([-(-n // _PAGE) for n in lens])
    total, widest = int(need.sum()), int(need.max())
    blocks = total + 7
    order = torch.randperm(blocks, generator=g, device="cuda")[:total].to(torch.int32)
    used = torch.arange(widest)[None] < need[:, None]
    bt = torch.full(used.shape, -1, dtype=torch.int32, device="cuda")
    bt[used.cuda()] = order
    return bt, blocks


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _masks(seed, counts, words, chain):
    """A random tree per sequence, node 0 its root (or a chain): each node's words name its ancestors and itself."""
    r = random.Random(seed)
    rows = []
    for n in counts:
        seen = []
        for i in range(n):
            parent = i - 1 if chain else r.randint(max(0, (i - 1) // 3 - 1), max(0, (i - 1) // 2))
            seen.append((seen[parent] if i else 0) | (1 << i))
        rows += [[_signed(m >> (64 * w) & (1 << 64) - 1) for w in range(words)] for m in seen]
    return torch.tensor(rows, dtype=torch.int64, device="cuda")


def _signed(u):
    return u - (1 << 64) if u >> 63 else u


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": dict(c), "scale": c["d"] ** -0.5, "kv_scale": _scale(c)}
    if c["op"] == "rope":
        t, dt = c["tokens"], _Q[c["q"]]
        blocks = -(-t // _PAGE) + 5
        s["q"] = _normal(g, t, c["hq"], c["d"], dtype=dt)
        s["key"] = _normal(g, t, c["hkv"], c["d"], dtype=dt)
        s["value"] = _normal(g, t, c["hkv"], c["d"], dtype=dt)
        s["q_out"] = torch.empty_like(s["q"])
        s["positions"] = torch.randint(0, c["far"], (t,), generator=g, device="cuda")
        s["slots"] = torch.randperm(blocks * _PAGE, generator=g, device="cuda")[:t]
        s["inv_freq"] = (500000.0 ** (-torch.arange(0, c["rot"], 2, dtype=torch.float64) / c["rot"])).float().cuda()
        s["k_cache"], s["v_cache"] = _pool(g, blocks, c), _pool(g, blocks, c)
        return s
    lens, counts = _lens(c)
    s["bt"], blocks = _tables(g, lens)
    s["k_cache"], s["v_cache"] = _pool(g, blocks, c), _pool(g, blocks, c)
    s["lens"] = _i32(lens)
    s["max_len"] = max(lens)
    if c["op"] == "commit":
        nodes = [c["nodes"]] * c["seqs"]
        # The nodes that move lie behind the places that paths move to, so a pass on the state that a pass left
        # moves the same rows again.
        r = random.Random(seed)
        path = [list(range(_kept(a))) + sorted(r.sample(range(a, c["nodes"]), a - _kept(a))) for a in counts]
        s["accepted"] = _i32([p + [-1] * (c["path"] - len(p)) for p in path])
        s["accepted_lens"] = _i32(counts)
        s["new_lens"] = torch.empty_like(s["lens"])
    else:
        nodes = counts
        q_dtype = torch.bfloat16 if c["kv"] == "e4m3" else _Q[c["kv"]]
        s["q"] = _normal(g, sum(nodes), c["hq"], c["d"], dtype=q_dtype)
        s["out"] = torch.empty_like(s["q"])
        s["mask"] = _masks(seed, nodes, -(-max(nodes) // 64), c["chain"])
        s["nodes"] = max(nodes)
        s["owner"] = torch.repeat_interleave(torch.arange(c["seqs"]), torch.tensor(nodes)).cuda()
        s["rank"] = torch.cat([torch.arange(n) for n in nodes]).cuda()
        s["workspace"] = torch.empty(160 << 20, dtype=torch.uint8, device="cuda")
    s["start"] = _i32([sum(nodes[:i]) for i in range(c["seqs"] + 1)])
    return s


def run(state):
    return {"rope": _run_rope, "tree": _run_tree, "commit": _run_commit}[state["case"]["op"]](state)


def _run_rope(s):
    c = s["case"]
    if own:
        import paged_kv_cache_385_b200 as pa
        pa.pa_rope_and_cache(s["q_out"], s["q"], s["key"], s["value"], s["positions"], s["inv_freq"], s["slots"],
                             s["k_cache"], s["v_cache"], interleaved=c["pairs"], k_scale=s["kv_scale"],
                             v_scale=s["kv_scale"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    angle = s["positions"].double()[:, None, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float(), angle.sin().float()
    s["q_out"].copy_(_rotate(s["q"].float(), cos, sin, c))
    _store(s["k_cache"], s["slots"], _rotate(s["key"].float(), cos, sin, c), s["kv_scale"])
    _store(s["v_cache"], s["slots"], s["value"].float(), s["kv_scale"])
    return s["q_out"], s["k_cache"], s["v_cache"]


def _rotate(x, cos, sin, c):
    turned, rest = x[..., :c["rot"]], x[..., c["rot"]:]
    if c["pairs"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        return torch.cat((torch.stack((a * cos - b * sin, b * cos + a * sin), dim=-1).flatten(-2), rest), dim=-1)
    a, b = turned.chunk(2, dim=-1)
    return torch.cat((a * cos - b * sin, b * cos + a * sin, rest), dim=-1)


def _store(pool, slots, rows, scale):
    if pool.dtype == torch.float8_e4m3fn:
        # Behind the largest finite value the cast gives NaN; a cache holds that value instead.
        pool = pool.view(torch.uint8)
        rows = (rows * (1.0 / scale)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    pool[slots // _PAGE, :, slots % _PAGE] = rows.to(pool.dtype)


def _run_tree(s):
    c = s["case"]
    if own:
        import paged_kv_cache_385_b200 as pa
        pa.pa_decode_tree(s["out"], s["q"], s["k_cache"], s["v_cache"], s["bt"], s["start"], s["lens"],
                          None if c["chain"] else s["mask"], s["nodes"], s["scale"], c["hkv"], softcap=c["cap"], k_scale=s["kv_scale"],
                          v_scale=s["kv_scale"], max_context_len=s["max_len"], workspace=s["workspace"])
        return s["out"]
    b, n, group, width = c["seqs"], s["nodes"], c["hq"] // c["hkv"], s["bt"].shape[1] * _PAGE
    pages = s["bt"].clamp(min=0).long()
    q = torch.zeros(b, n, c["hkv"], group, c["d"], device="cuda")
    q[s["owner"], s["rank"]] = s["q"].float().unflatten(1, (c["hkv"], group))
    q = q.permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seqs, kv heads, nodes * group, d]
    keys = s["k_cache"].view(torch.uint8)[pages].view(s["k_cache"].dtype).transpose(1, 2).flatten(2, 3).float()
    scores = (q @ keys.transpose(-1, -2)).mul_(s["scale"] * s["kv_scale"])
    del keys
    if c["cap"]:
        scores = scores.div_(c["cap"]).tanh_().mul_(c["cap"])
    # A node sees the whole context before the tree, and the nodes that its mask names.
    first = s["lens"] - (s["start"][1:] - s["start"][:-1])
    at = torch.arange(width, device="cuda") - first[:, None]  # [seqs, width]: the node held there
    word = (at // 64).clamp(0, s["mask"].shape[1] - 1)
    masks = torch.zeros(b, n, s["mask"].shape[1], dtype=torch.int64, device="cuda")
    masks[s["owner"], s["rank"]] = s["mask"]
    bits = masks.gather(2, word[:, None].expand(b, n, width)) >> (at % 64)[:, None] & 1
    seen = (at < 0)[:, None] | (bits > 0) & (at[:, None] < (s["lens"] - first)[:, None, None])
    scores = scores.unflatten(2, (n, group)).masked_fill_(~seen[:, None, :, None], -math.inf).flatten(2, 3)
    top = scores.amax(dim=-1, keepdim=True)
    weights = scores.sub_(torch.where(top.isinf(), 0.0, top)).exp_()
    total = weights.sum(dim=-1, keepdim=True)
    held = (torch.arange(width, device="cuda") < s["lens"][:, None])[:, None, :, None]
    values = s["v_cache"].view(torch.uint8)[pages].view(s["v_cache"].dtype).transpose(1, 2).flatten(2, 3).float()
    out = (weights @ values.masked_fill_(~held, 0.0)) * (s["kv_scale"] / total.masked_fill(total == 0, 1.0))
    out = out.unflatten(2, (n, group)).permute(0, 2, 1, 3, 4).flatten(2, 3)  # [seqs, nodes, heads, d]
    s["out"].copy_(out[s["owner"], s["rank"]])
    return s["out"]


def _run_commit(s):
    if own:
        import paged_kv_cache_385_b200 as pa
        pa.pa_commit_tree(s["k_cache"], s["v_cache"], s["bt"], s["start"], s["lens"], s["accepted"],
                          s["accepted_lens"], s["new_lens"])
        return s["k_cache"], s["v_cache"], s["new_lens"]
    first = (s["lens"] - (s["start"][1:] - s["start"][:-1]))[:, None].long()
    to = torch.arange(s["accepted"].shape[1], device="cuda").expand_as(s["accepted"])
    taken = to < s["accepted_lens"][:, None]
    src = _slot(s["bt"], first + torch.where(taken, s["accepted"], 0))
    dst = _slot(s["bt"], first + torch.where(taken, to, 0))  # what is not accepted: the root, onto itself
    _move(s["k_cache"], src, dst)
    _move(s["v_cache"], src, dst)
    s["new_lens"].copy_(first[:, 0] + s["accepted_lens"])
    return s["k_cache"], s["v_cache"], s["new_lens"]


def _slot(bt, at):
    return (bt.gather(1, at // _PAGE) * _PAGE + at % _PAGE).flatten()


def _move(pool, src, dst):
    pool = pool.view(torch.uint8)
    pool[dst // _PAGE, :, dst % _PAGE] = pool[src // _PAGE, :, src % _PAGE]


def exact(case, seed):
    """What the operators are defined as, in 64 bits, sequence by sequence and row by row."""
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rope(s, case)
    lens, counts = _lens(case)
    k, v = s["k_cache"].double(), s["v_cache"].double()
    if case["op"] == "commit":
        for i, (n, a) in enumerate(zip(lens, counts)):
            base = n - case["nodes"]
            table, path = s["bt"][i].tolist(), s["accepted"][i].tolist()
            for to, node in enumerate(path[:a]):
                p, r = base + node, base + to
                for pool in (k, v):
                    pool[table[r // _PAGE], :, r % _PAGE] = pool[table[p // _PAGE], :, p % _PAGE]
        return k, v, torch.tensor([n - case["nodes"] + a for n, a in zip(lens, counts)], dtype=torch.int32)
    del k, v
    out, row = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), 0
    group = case["hq"] // case["hkv"]
    words = s["mask"].tolist()
    for i, (n, nodes) in enumerate(zip(lens, counts)):
        table = s["bt"][i, :-(-n // _PAGE)].long()
        named = [[words[row + a][b // 64] >> (b % 64) & 1 for b in range(nodes)] for a in range(nodes)]
        seen = torch.ones(nodes, n, dtype=torch.bool, device="cuda")
        seen[:, n - nodes:] = torch.tensor(named, device="cuda") > 0
        for h in range(case["hkv"]):
            k = s["k_cache"][table, h].double().reshape(-1, case["d"])[:n] * s["kv_scale"]
            v = s["v_cache"][table, h].double().reshape(-1, case["d"])[:n] * s["kv_scale"]
            q = s["q"][row:row + nodes, h * group:(h + 1) * group].double()
            x = torch.einsum("agd,td->gat", q, k) / math.sqrt(case["d"])
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            p = torch.softmax(x.masked_fill(~seen, -math.inf), dim=-1).nan_to_num(0.0)
            out[row:row + nodes, h * group:(h + 1) * group] = torch.einsum("gat,td->agd", p, v)
        row += nodes
    return out


def _exact_rope(s, case):
    rot = case["rot"]
    d = torch.arange(rot, device="cuda")
    pair = d // 2 if case["pairs"] else d % (rot // 2)
    first = d % 2 == 0 if case["pairs"] else d < rot // 2
    mate = torch.where(first, d + 1, d - 1) if case["pairs"] else (d + rot // 2) % rot
    sign = torch.where(first, -1.0, 1.0).double()
    angle = s["positions"].double()[:, None] * s["inv_freq"].double()[pair]

    def turned(x):
        y = x.double().clone()
        y[..., :rot] = x[..., :rot].double() * angle.cos()[:, None] + sign * x[..., mate].double() * angle.sin()[:, None]
        return y

    def stored(pool, rows):
        pool = pool.double()
        if case["kv"] == "e4m3":  # what a cache of codes stands for, before it is rounded
            rows = (rows / s["kv_scale"]).clamp(-448.0, 448.0)
        pool[s["slots"] // _PAGE, :, s["slots"] % _PAGE] = rows
        return pool

    return turned(s["q"]), stored(s["k_cache"], turned(s["key"])), stored(s["v_cache"], s["value"].double())
