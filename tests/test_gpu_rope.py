"""pa_rope_and_cache on the GPU against the float64 definition (oracle/tree.py) and the oracle's scatter."""
import numpy as np
import pytest
import torch

import paged_kv_cache_385_b200 as pa
from oracle import cache, e4m3, tree

pytestmark = pytest.mark.gpu

KV = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(autouse=True)
def _no_device_error():
    pa.pa_read_device_error(clear=True)
    yield
    assert pa.pa_read_device_error(clear=True) == 0


class RopeCase:
    def __init__(self, src, kv, d, rot, hq, hkv, tokens, pairs=False, far=4096, seed=1, magnitude=1.0, skip=()):
        g = torch.Generator().manual_seed(seed)
        self.dt, self.kv, self.pairs, self.magnitude = {"f16": torch.float16, "bf16": torch.bfloat16}[src], kv, pairs, magnitude
        self.src = src
        self.q, self.k, self.v = (torch.randn(tokens, h, d, generator=g).to(self.dt) for h in (hq, hkv, hkv))
        self.pos = torch.randint(0, far, (tokens,), generator=g)
        self.inv = pa.pa_rope_inv_freq(rot, 500000.0)
        blocks = tokens // 16 + 3
        self.slots = torch.randperm(blocks * 16, generator=g)[:tokens]
        for i in skip:
            self.slots[i] = -1
        elem = 1 if kv == "e4m3" else 2
        self.sentinel = [torch.randint(0, 256, (blocks, hkv, 16, d * elem), generator=g, dtype=torch.uint8) for _ in range(2)]
        self.ks, self.vs = (0.011, 0.02) if kv == "e4m3" else (1.0, 1.0)

    def run(self, in_place=False, no_q=False, stream=None):
        self.kc, self.vc = (s.cuda().view(KV[self.kv]) for s in self.sentinel)
        q = self.q.cuda()
        out = q if in_place else torch.full_like(q, 77.0)
        pa.pa_rope_and_cache(None if no_q else out, None if no_q else q, self.k.cuda(), self.v.cuda(), self.pos.cuda(),
                             self.inv.cuda(), self.slots.cuda(), self.kc, self.vc, interleaved=self.pairs,
                             magnitude=self.magnitude, k_scale=self.ks, v_scale=self.vs, stream=stream)
        torch.cuda.synchronize()
        return out

    def near(self, got, x, want, u):
        """got within one rounding (u, relative) of want, and the sines' and products' float32 errors: each
        product is off by 2^-24 (the operand's) + 2^-24 (its own rounding) + 2^-21.9 (the angle's and
        sine's), of |x| + |y| at most, so 2^-20 of a pair's size covers the sum of both."""
        pair = np.abs(x).max(axis=-1, keepdims=True) * self.magnitude * 2
        err = np.abs(got - want)
        assert np.all(err <= u * np.abs(want) * (1 + 2.0 ** -7) + 2.0 ** -20 * pair), err.max()

    def check(self, out):
        rot = 2 * len(self.inv)
        x = self.q.double().numpy()
        want = tree.rotate(x, self.pos.numpy(), self.inv.numpy(), self.pairs, self.magnitude)
        u = 2.0 ** -11 if self.dt == torch.float16 else 2.0 ** -8
        if out is not None:
            self.near(out.double().cpu().numpy(), x, want, u)
            assert torch.equal(out[..., rot:].cpu(), self.q[..., rot:])
        k = self.k.double().numpy()
        k_want = tree.rotate(k, self.pos.numpy(), self.inv.numpy(), self.pairs, self.magnitude)
        got_k, got_v = (c.view(torch.uint8).cpu().numpy() for c in (self.kc, self.vc))
        if self.kv == "e4m3":
            v_rows = self.v.float().numpy()
        else:
            v_rows = self.v.view(torch.int16).numpy().view(np.uint16)
        empty = [s.numpy() for s in self.sentinel]
        # Values (and every byte that nobody writes) are the oracle's scatter, bit for bit.
        _, v_pool = cache.reshape_and_cache(v_rows, v_rows, self.slots.numpy(), empty[1], empty[1], self.kv, self.vs, self.vs)
        assert np.array_equal(got_v, v_pool)
        written = np.zeros(got_k.shape[:3], dtype=bool)
        for t, slot in enumerate(self.slots.tolist()):
            if slot < 0:
                continue
            written[slot // 16, :, slot % 16] = True
            row = got_k[slot // 16, :, slot % 16]
            if self.kv == "e4m3":
                y = k_want[t] / np.float64(np.float32(self.ks))
                got = e4m3.decode(row)
                # One e4m3 rounding of a value that float32 holds to 2^-20 of the pair: half a step is 2^-4 of
                # a normal value and 2^-10 below 2^-6.
                err = np.abs(got - np.clip(y, -448, 448))
                pair = np.abs(k[t]).max() / self.ks * self.magnitude * 2
                assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(y), 2.0 ** -10) + 2.0 ** -20 * pair)
            else:
                got = cache.pool_values(row, self.kv)
                self.near(got[None], k[t][None], k_want[t][None], u)
                assert np.array_equal(row.view(np.uint16)[:, rot:], self.k[t].view(torch.int16).numpy().view(np.uint16)[:, rot:])
        assert np.array_equal(got_k[~written], empty[0][~written])


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("src,kv", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("d,rot", [(128, 128), (128, 64), (64, 64), (128, 24), (64, 8), (96, 24), (80, 32), (8, 8), (24, 16)])
def test_against_the_definition(src, kv, d, rot, pairs):
    c = RopeCase(src, kv, d, rot, hq=6, hkv=2, tokens=21, pairs=pairs, seed=d + rot, skip=(3, 20))
    c.check(c.run())


@pytest.mark.parametrize("tokens", [1, 2, 16, 300])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (32, 8), (7, 7)])
def test_token_and_head_counts(tokens, hq, hkv):
    c = RopeCase("bf16", "bf16", 128, 128, hq, hkv, tokens, seed=tokens)
    c.check(c.run())


@pytest.mark.parametrize("pairs", [False, True])
def test_far_and_negative_positions(pairs):
    """Angles of a million radians and more are those of the float64 product."""
    c = RopeCase("f16", "f16", 64, 64, 2, 1, 6, pairs=pairs)
    c.pos = torch.tensor([0, -5, 10 ** 6 + 1, 2 ** 28 + 7, -(10 ** 7), 131071])
    c.check(c.run())


def test_in_place_and_without_queries():
    c = RopeCase("bf16", "bf16", 128, 64, 4, 2, 33, seed=4)
    out = c.run()
    assert torch.equal(c.run(in_place=True), out)
    c.check(out)
    c.run(no_q=True)
    c.check(None)


def test_magnitude_and_stream():
    c = RopeCase("f16", "e4m3", 128, 128, 4, 2, 40, seed=5, magnitude=1.25)
    side = torch.cuda.Stream()
    c.check(c.run(stream=side))


def test_zero_position_is_the_plain_write():
    """At position 0 nothing turns: the pools are pa_reshape_and_cache's, byte for byte."""
    for kv in ("bf16", "e4m3"):
        c = RopeCase("bf16", kv, 128, 128, 2, 2, 50, seed=6, skip=(7,))
        c.pos.zero_()
        out = c.run()
        assert torch.equal(out.cpu(), c.q)
        kc, vc = (s.cuda().view(KV[kv]) for s in c.sentinel)
        pa.pa_reshape_and_cache(c.k.cuda(), c.v.cuda(), c.slots.cuda(), kc, vc, c.ks, c.vs)
        assert torch.equal(c.kc.view(torch.uint8), kc.view(torch.uint8))
        assert torch.equal(c.vc.view(torch.uint8), vc.view(torch.uint8))


def test_strided_rows():
    """Queries, keys and values as views of one packed projection, the queries rotated in place."""
    c = RopeCase("bf16", "bf16", 128, 128, 4, 2, 20, seed=7)
    want = c.run()
    kc, vc = c.kc.clone(), c.vc.clone()
    qkv = torch.cat((c.q, c.k, c.v), dim=1).cuda()
    c.kc, c.vc = (s.cuda().view(torch.bfloat16) for s in c.sentinel)
    pa.pa_rope_and_cache(qkv[:, :4], qkv[:, :4], qkv[:, 4:6], qkv[:, 6:], c.pos.cuda(), c.inv.cuda(), c.slots.cuda(), c.kc, c.vc)
    assert torch.equal(qkv[:, :4], want) and torch.equal(qkv[:, 4:].cpu(), torch.cat((c.k, c.v), dim=1))
    assert torch.equal(c.kc.view(torch.int16), kc.view(torch.int16)) and torch.equal(c.vc.view(torch.int16), vc.view(torch.int16))


def test_slots_outside_the_pool():
    c = RopeCase("f16", "f16", 64, 64, 2, 1, 5, seed=8)
    want = c.run()
    word = torch.zeros(1, dtype=torch.int32, device="cuda")
    slots = c.slots.clone()
    slots[1], slots[3] = c.kc.shape[0] * 16, -2
    kc, vc = (s.cuda().view(torch.float16) for s in c.sentinel)
    out = torch.empty_like(want)
    pa.pa_rope_and_cache(out, c.q.cuda(), c.k.cuda(), c.v.cuda(), c.pos.cuda(), c.inv.cuda(), slots.cuda(), kc, vc, error_word=word)
    assert int(word) == pa.PA_DEVERR_BAD_SLOT
    assert torch.equal(out, want)
    c.kc, c.vc, c.slots = kc, vc, torch.where((slots < 0) | (slots >= kc.shape[0] * 16), -1, slots)
    c.check(out)
