"""Prompt and page operators on the GPU (isd_chunk_attention, isd_fork_requests,
isd_compact_pages) against oracle.cache_oracle in 64 bits.

Tolerance of an attention output, per element: the weights p are rounded to
bf16 before the product with V (half a step, 2^-8 of sum p|v|) and the result
once more (2^-8 of itself).  A score is a sum of D fp32 products, off by at most
(D + 8) 2^-23 of sum |q k| * scale, which moves numerator and denominator by as
much each; sums over the keys are fp32 in chunks of at least 8 (keys / 8 steps
of 2^-23, and 2^-14 covers the exponential and the merging of partial sums).
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import cache_oracle as O

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def isd():
    from speculative_verification_isd_b200 import isd as lib
    return lib


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


class Chunk:
    """A chunk call's buffers: pages in random order, NaN in every cache row
    that no request has, sentinels in the rows of no request."""

    def __init__(self, isd, Hq, Hkv, D, P, ctx, n, seed=0, before=0, after=0, scale=0.0, gain=1.0):
        self.isd = isd
        rng = np.random.default_rng(seed)
        B = len(ctx)
        self.ctx, self.n = list(ctx), list(n)
        used = [-(-(c + m) // P) for c, m in zip(ctx, n)]
        cols, pages = max(max(used), 1) + 1, sum(used) + 3
        perm = rng.permutation(pages)
        table = np.full((B, cols), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = perm[at:at + u]
            at += u
        self.T = T = before + sum(n) + after
        self.start = [before + sum(n[:b]) for b in range(B + 1)]
        self.q, self.k_new, self.v_new = bf16(rng, T, Hq, D) * gain, bf16(rng, T, Hkv, D), bf16(rng, T, Hkv, D)
        nan = float("nan")
        for t in list(range(before)) + list(range(T - after, T)):
            self.q[t], self.k_new[t], self.v_new[t] = nan, nan, nan
        self.k_pool = torch.full((pages, P, Hkv, D), nan, dtype=torch.bfloat16)
        self.v_pool = self.k_pool.clone()
        for b, c in enumerate(ctx):
            pos = np.arange(c)
            for pool in (self.k_pool, self.v_pool):
                pool[table[b, pos // P], pos % P] = bf16(rng, c, Hkv, D)
        self.table = table
        self.dims = isd.make_dims(B, 1, Hq, Hkv, D, 1, P, pages, cols, sm_scale=scale) if scale else \
            isd.make_dims(B, 1, Hq, Hkv, D, 1, P, pages, cols)
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def upload(self):
        self.d_in = [x.cuda() for x in (self.q, self.k_new, self.v_new)]
        self.d_pool = [x.cuda() for x in (self.k_pool, self.v_pool)]
        self.d_idx = [i32(self.table), i32(self.ctx), i32(self.start)]
        self.out = torch.full((self.T, self.dims.Hq * self.dims.D), 7.0, dtype=torch.bfloat16, device="cuda")
        self.ws = self.isd.alloc_chunk_workspace(self.dims, self.T)
        self.ws.fill_(0xA5)   # no initial contents are required
        return self

    def call(self, **kw):
        self.isd.chunk_attention(self.dims, *self.d_in, *self.d_pool, *self.d_idx, self.out, self.ws, self.err, **kw)
        return self

    def check(self, flags=0):
        torch.cuda.synchronize()
        assert int(self.err.item()) == flags
        d = self.dims
        kp = O.append(f64(self.k_pool), f64(self.k_new), self.table, self.ctx, self.start)
        vp = O.append(f64(self.v_pool), f64(self.v_new), self.table, self.ctx, self.start)
        for got, want in zip(self.d_pool, (kp, vp)):
            assert np.array_equal(f64(got), want, equal_nan=True)
        want, weight, reach = O.chunk_attention(f64(self.q), kp, vp, self.table, self.ctx, self.start, d.sm_scale)
        check_rows(f64(self.out).reshape(want.shape), want, weight, reach, d.D,
                   max(c + m for c, m in zip(self.ctx, self.n)))
        return self


def check_rows(got, want, weight, reach, D, keys):
    """Rows with a value within the tolerance; rows of no request (want is NaN
    and weight is NaN) still hold the sentinel; non-finite values alike."""
    mine = ~np.isnan(weight).all(axis=(1, 2)) | (reach > 0).any(axis=(1, 2))
    assert (got[~mine] == 7.0).all()
    got, want, weight, reach = got[mine], want[mine], weight[mine], reach[mine]
    ok = np.isfinite(want)
    assert np.array_equal(got[~ok], want[~ok], equal_nan=True)
    assert np.isfinite(got[ok]).all()
    tol = 2.0 ** -8 * (weight + np.abs(want)) + \
        (2 * (D + 8) * 2.0 ** -23 * reach + keys / 8 * 2.0 ** -23 + 2.0 ** -14) * weight + 1e-30
    bad = np.abs(got[ok] - want[ok]) / tol[ok]
    assert bad.size == 0 or bad.max() <= 1, bad.max()


SHAPES = {
    # name: Hq, Hkv, D, P, cached lengths, new tokens
    "one_token_no_prefix": (4, 1, 128, 16, [0], [1]),
    "decode": (8, 2, 128, 16, [1000, 0, 1, 127, 128, 129, 255, 16], [1] * 8),
    "decode_d64": (14, 2, 64, 24, [7, 500, 0, 128], [1] * 4),
    "decode_long": (8, 2, 128, 64, [20001, 3], [1, 1]),
    "prompt": (8, 2, 128, 16, [0], [333]),
    "prompt_d64": (6, 2, 64, 16, [0, 0], [129, 256]),
    "mixed": (8, 2, 128, 16, [0, 700, 128, 1, 64, 0], [200, 1, 128, 0, 65, 31]),
    "all_empty_but_one": (4, 2, 128, 8, [0, 50, 0, 9], [0, 0, 3, 0]),
    "few_rows": (4, 1, 128, 32, [300, 120, 128, 5], [2, 8, 9, 16]),
    "page_1": (4, 2, 128, 1, [40, 200], [7, 1]),
    "page_5": (4, 1, 64, 5, [131, 0], [4, 20]),
    "page_24": (7, 1, 64, 24, [250, 23], [40, 3]),
    "page_100": (4, 2, 128, 100, [399, 100], [30, 1]),
    "page_256": (4, 1, 128, 256, [500, 130], [140, 2]),
    "one_head_per_group": (3, 3, 128, 16, [77, 300], [150, 1]),
    "group_3": (9, 3, 64, 16, [200, 0], [90, 1]),
    "group_7": (28, 4, 128, 16, [150, 90], [41, 1]),
    "group_8": (64, 8, 128, 16, [130, 1], [20, 1]),
    "group_128": (128, 1, 128, 16, [130, 7], [3, 1]),
    "group_100": (100, 1, 64, 16, [140, 0], [3, 2]),
    "remainders": (5, 1, 128, 16, [36, 52, 40, 37], [255, 303, 204, 302]),
    "remainders_d64": (3, 1, 64, 8, [20, 70, 100], [258, 513, 389]),
    "split_rows": (8, 2, 128, 16, [9000], [70]),
    "many_requests": (4, 2, 128, 16, [(37 * i) % 300 for i in range(90)], [(5 * i) % 4 for i in range(90)]),
}


@pytest.mark.parametrize("name", SHAPES)
def test_chunk(isd, name):
    Hq, Hkv, D, P, ctx, n = SHAPES[name]
    c = Chunk(isd, Hq, Hkv, D, P, ctx, n, seed=len(name), before=2 if len(ctx) > 1 else 0, after=5)
    c.upload().call().check()


# enough work that every CTA walks several items of many key tiles
LONG = {
    "decode_long_pieces": (8, 8, 128, 16, [(613 * i) % 2900 for i in range(40)], [1] * 40),
    "decode_d64_long_pieces": (16, 8, 64, 32, [(613 * i) % 2900 for i in range(40)], [1 + i % 3 for i in range(40)]),
    "prompt_long_pieces": (16, 8, 64, 16, [0, 900], [900, 700]),
    "prompt_d128_long_pieces": (32, 8, 128, 16, [300], [1100]),
    "mixed_long_pieces": (8, 4, 128, 24, [(389 * i) % 2100 for i in range(30)],
                          [1 if i % 3 else 40 + 9 * i for i in range(30)]),
}


def test_chunk_one_key_is_its_value(isd):
    """A row with one key is that key's value to the last bit."""
    c = Chunk(isd, 8, 2, 128, 16, [0] * 5, [1, 1, 3, 1, 20], seed=2, gain=7.0).upload().call().check()
    first = [c.start[b] for b in range(5)]
    got = c.out.view(-1, 8, 128)[first]
    assert torch.equal(got, c.d_in[2][first].repeat_interleave(4, 1))


def test_chunk_more_requests_than_threads(isd):
    """The cut of the work goes over the requests in several rounds, twice."""
    B = 900
    ctx = [(7 * b) % 90 for b in range(B)]
    n = [0 if b % 3 else 1 + b % 2 for b in range(B)]
    n[-1], ctx[-1] = 40, 300
    Chunk(isd, 4, 2, 64, 16, ctx, n, seed=5, after=3).upload().call().check()


def test_chunk_one_long_request_many_parts(isd):
    """One KV head over a long context: the item is cut between all CTAs."""
    Chunk(isd, 8, 1, 128, 64, [30011], [2], seed=6).upload().call().check()
    Chunk(isd, 4, 1, 64, 16, [18000], [20], seed=7).upload().call().check()


def test_chunk_piece_of_seconds(isd):
    """A piece of 2^22 tiles per CTA (2.6 s): no wait gives up while the others go
    on.  The requests' pages are one and the same; scores 0 and values 1 make every
    sum a whole number that 32 bits hold, and the result 1."""
    kv, P, D = (1 << 29) + 5, 1024, 64
    B = torch.cuda.get_device_properties(0).multi_processor_count
    cols = kv // P + 1
    table = torch.zeros(B, cols, dtype=torch.int32, device="cuda")
    table[:, -1] = torch.arange(1, B + 1, dtype=torch.int32, device="cuda")   # the new tokens' own pages
    zeros, ones = (torch.full((B + 1, P, 1, D), x, dtype=torch.bfloat16, device="cuda") for x in (0.0, 1.0))
    q = bf16(np.random.default_rng(1), B, 1, D).cuda()
    d = isd.make_dims(B, 1, 1, 1, D, 1, P, B + 1, cols)
    out, err = torch.zeros(B, D, dtype=torch.bfloat16, device="cuda"), i32([0])
    isd.chunk_attention(d, q, torch.zeros_like(q), torch.ones_like(q), zeros, ones, table, i32([kv] * B),
                        i32(np.arange(B + 1)), out, isd.alloc_chunk_workspace(d, B), err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    assert (out == 1).all()


@pytest.mark.parametrize("gain", [1.0, 20.0])
@pytest.mark.parametrize("name", LONG)
def test_chunk_long_pieces(isd, name, gain):
    Hq, Hkv, D, P, ctx, n = LONG[name]
    Chunk(isd, Hq, Hkv, D, P, ctx, n, seed=3, gain=gain).upload().call().check()


@pytest.mark.parametrize("n", [1, 40])
def test_chunk_rising_scores_long_pieces(isd, n):
    """The running maximum moves in every tile of pieces of many tiles."""
    B, kv = 20, 1500
    c = Chunk(isd, 8, 8, 128, 16, [kv] * B, [n] * B, seed=9)
    c.q[:] = 1.0
    ramp = (torch.arange(kv + n, dtype=torch.float32) / 64)[:, None, None].expand(-1, 8, 128).to(torch.bfloat16)
    pos = np.arange(kv)
    for b in range(B):
        c.k_pool[c.table[b, pos // 16], pos % 16] = ramp[:kv]
        c.k_new[b * n:(b + 1) * n] = ramp[kv:]
    c.upload().call().check()


def test_chunk_hidden_keys_long_pieces(isd):
    """Non-finite values noted for one item do not reach the next ones."""
    ctx, n = [700, 0, 300, 50] * 10, [30, 300, 3, 90] * 10
    c = Chunk(isd, 8, 4, 64, 16, ctx, n, seed=21)
    rng = np.random.default_rng(1)
    odd = torch.tensor([float("nan"), float("inf"), float("-inf")])
    for t in rng.integers(0, sum(n), 60):
        c.v_new[t, rng.integers(0, 4), rng.integers(0, 64)] = odd[rng.integers(0, 3)]
    c.upload().call().check()


@pytest.mark.parametrize("gain,scale", [(30.0, 0.0), (1.0, 0.5), (1.0, 1e-3)])
def test_chunk_scores_far_apart(isd, gain, scale):
    """Row maxima that move by more than 2^8 between tiles; flat scores."""
    Chunk(isd, 8, 2, 128, 16, [600, 3], [40, 300], seed=5, gain=gain, scale=scale).upload().call().check()


def test_chunk_rising_scores(isd):
    """Every key beats the ones before it: the maximum moves in every tile."""
    c = Chunk(isd, 4, 1, 128, 16, [1500], [64], seed=9)
    c.q[:] = 1.0
    ramp = torch.arange(1564, dtype=torch.float32) / 64
    pos = np.arange(1500)
    c.k_pool[c.table[0, pos // 16], pos % 16] = ramp[:1500, None, None].expand(-1, 1, 128).to(torch.bfloat16)
    c.k_new[:64] = ramp[1500:, None, None].expand(-1, 1, 128).to(torch.bfloat16)
    c.upload().call().check()


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_chunk_hidden_keys_do_not_reach(isd, value):
    """A non-finite key or value changes only the rows that see it."""
    c = Chunk(isd, 4, 2, 128, 16, [100, 20, 0, 300], [150, 40, 200, 3], seed=3)
    c.v_new[60, 0, 5] = value
    c.v_new[149, 1, 127] = value
    c.k_new[120, 0, 64] = value if value != value else 0.0
    c.v_new[150 + 39, 0, 0] = value
    c.v_new[190 + 70, 1, 64] = value
    c.v_new[190 + 130, 1, 3] = value
    c.v_new[390 + 1, 0, 9] = value
    c.upload().call().check()


def test_chunk_opposite_infinities(isd):
    c = Chunk(isd, 4, 2, 128, 16, [0, 10], [200, 6], seed=4)
    c.v_new[20, 0, 5], c.v_new[90, 0, 5] = float("inf"), float("-inf")
    c.v_new[201, 1, 7], c.v_new[203, 1, 7] = float("-inf"), float("inf")
    c.upload().call().check()


@pytest.mark.parametrize("heads,ctx,n", [((8, 2, 128), [5000, 10, 300], [30, 200, 1]),
                                         ((28, 4, 128), [(701 * i) % 3000 for i in range(20)],
                                          [1 + (7 * i) % 40 for i in range(20)])])
def test_chunk_repeats_bit_for_bit(isd, heads, ctx, n):
    """Also where rows of a tile are no one's, whatever other calls left behind
    on the chip meanwhile."""
    c = Chunk(isd, *heads, 16, ctx, n, seed=6).upload().call()
    other = Chunk(isd, *heads, 16, [900] * 6, [70, 3, 20, 1, 9, 130], seed=7, gain=30.0).upload()
    first = c.out.clone()
    for _ in range(4):
        other.call()
        c.out.fill_(3.0)
        c.call()
        torch.cuda.synchronize()
        assert torch.equal(c.out.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("n", [1, 2, 40, 90])
@pytest.mark.parametrize("first", [100, 200, 390])
def test_chunk_first_scores_are_minus_infinity(isd, n, first):
    """Keys of score -inf count for nothing, also where they are a row's first
    tiles: the rows are the attention over the keys after them."""
    B, kv = 12, 400
    c = Chunk(isd, 8, 8, 128, 16, [kv] * B, [n] * B, seed=first + n)
    c.q[:] = c.q.abs() + 0.125
    pos = np.arange(kv)
    for b in range(B):
        c.k_pool[c.table[b, pos[:first] // 16], pos[:first] % 16] = float("-inf")
    c.upload().call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    kp = O.append(f64(c.k_pool), f64(c.k_new), c.table, c.ctx, c.start)
    vp = O.append(f64(c.v_pool), f64(c.v_new), c.table, c.ctx, c.start)
    got = f64(c.out).reshape(-1, 8, 128)
    for b in range(B):
        k, v = (O.rows_of(x, c.table[b], kv + n)[first:] for x in (kp, vp))
        q = f64(c.q)[c.start[b]:c.start[b + 1]]
        want = O.chunk_attention(q, k[:, None], v[:, None], [list(range(kv + n - first))], [kv - first], [0, n],
                                 c.dims.sm_scale)
        check_rows(got[c.start[b]:c.start[b + 1]], *want, 128, kv + n)


def test_chunk_in_pieces_is_the_whole(isd):
    """A prompt in pieces fills the same cache; its last rows agree with the
    prompt at once within both calls' tolerances."""
    whole = Chunk(isd, 8, 2, 128, 16, [0], [301], seed=8).upload().call().check()
    d, at = whole.dims, 0
    pools = [torch.full_like(p, float("nan")) for p in whole.d_pool]
    for n in (128, 1, 100, 72):
        out = torch.empty(n, d.Hq * d.D, dtype=torch.bfloat16, device="cuda")
        sl = [x[at:at + n].contiguous() for x in whole.d_in]
        isd.chunk_attention(d, *sl, *pools, whole.d_idx[0], i32([at]), i32([0, n]), out,
                            isd.alloc_chunk_workspace(d, n), whole.err)
        w = whole.out[at:at + n].float()
        assert (out.float() - w).abs().max().item() <= 4 * 2.0 ** -8 * whole.v_new.float().abs().max().item()
        at += n
    for a, b in zip(pools, whole.d_pool):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_chunk_bad_page_reads_zeros(isd):
    c = Chunk(isd, 4, 2, 128, 16, [200, 40], [20, 3], seed=10)
    c.table[0, 3] = 10 ** 6
    c.table[1, 1] = -5
    c.upload().call().check(isd.FLAG_PAGE_OOB)


BAD_PAGES = {
    # name: Hq, Hkv, D, P, cached lengths, new tokens, (request, column) of the pages outside the pool
    "in_the_last_cached_tile": (8, 2, 128, 4, [100, 33], [9, 1], [(0, 26), (1, 8)]),
    "in_the_last_cached_tile_d64": (6, 2, 64, 8, [40, 3], [16, 2], [(0, 6), (1, 0)]),
    "one_token": (4, 1, 128, 16, [128, 0, 64], [1, 1, 1], [(0, 8), (1, 0), (2, 4)]),
    "tiles": (8, 2, 128, 16, [0, 200], [300, 70], [(0, 1), (0, 10), (1, 14)]),
    "tiles_d64": (6, 2, 64, 24, [130, 0], [170, 400], [(0, 6), (0, 12), (1, 0), (1, 16)]),
    "page_1": (4, 2, 64, 1, [5, 0], [200, 20], [(0, 3), (0, 5), (0, 100), (0, 204), (1, 19)]),
    "page_3": (4, 1, 128, 3, [1], [300], [(0, 41), (0, 42), (0, 99)]),
    "page_100": (4, 2, 128, 100, [150], [300], [(0, 2), (0, 4)]),
    "page_256": (4, 1, 128, 256, [500], [140], [(0, 2)]),
    "group_100": (100, 1, 64, 16, [140, 0], [30, 2], [(0, 9), (1, 0)]),
    "long": (8, 4, 128, 16, [3000, 10], [700, 900], [(0, 200), (0, 231), (1, 30)]),
}


@pytest.mark.parametrize("name", BAD_PAGES)
def test_chunk_new_tokens_on_bad_pages_are_zeros(isd, name):
    """What a page outside the pool would hold counts as zeros for the tokens
    that the call appends as it does for the cached ones, whatever they are."""
    Hq, Hkv, D, P, ctx, n, bad = BAD_PAGES[name]
    c = Chunk(isd, Hq, Hkv, D, P, ctx, n, seed=31)
    for k, (b, col) in enumerate(bad):
        c.table[b, col] = (-2, 10 ** 6, c.dims.num_pages)[k % 3]
        for i in range(max(0, col * P - ctx[b]), min(n[b], (col + 1) * P - ctx[b])):
            c.k_new[c.start[b] + i], c.v_new[c.start[b] + i] = float("nan"), float("nan")
    c.upload().call().check(isd.FLAG_PAGE_OOB)


@pytest.mark.parametrize("what", ["negative", "over"])
def test_chunk_capacity(isd, what):
    c = Chunk(isd, 4, 2, 128, 16, [50, 60, 70], [20, 5, 30], seed=11).upload()
    keep = [p.clone() for p in c.d_pool]
    c.d_idx[1][1] = -1 if what == "negative" else c.dims.max_pages_per_req * 16 - 2
    c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == isd.FLAG_CAPACITY
    out = c.out.clone()
    assert (out[20:25] == 0).all()
    # the other requests are served as ever, and this one's pages keep their bytes
    c.d_idx[1].copy_(i32(c.ctx))
    for p, k in zip(c.d_pool, keep):
        mine = c.d_idx[0][1, :5].long()
        assert torch.equal(p[mine].view(torch.int16), k[mine].view(torch.int16))
    c.err.zero_()
    c.call().check()
    assert torch.equal(out[:20], c.out[:20]) and torch.equal(out[25:], c.out[25:])


@pytest.mark.parametrize("starts", [[0, 9, 5, 12], [-1, 3, 5, 12], [0, 3, 5, 13]])
def test_chunk_range(isd, starts):
    c = Chunk(isd, 4, 2, 128, 16, [10, 20, 30], [3, 2, 7], seed=12).upload()
    keep = [p.clone() for p in c.d_pool]
    c.d_idx[2] = i32(starts)
    c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == isd.FLAG_CHUNK_RANGE
    assert (c.out == 7).all()
    for p, k in zip(c.d_pool, keep):
        assert torch.equal(p.view(torch.int16), k.view(torch.int16))


def test_chunk_graph_and_streams(isd):
    """Captured and replayed with other lengths; two calls on two streams at
    once, each with its workspace."""
    a = Chunk(isd, 8, 2, 128, 16, [400, 90, 0], [40, 1, 100], seed=13).upload()
    b = Chunk(isd, 8, 2, 128, 16, [3000, 20], [1, 90], seed=14).upload()
    a.call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a.call()
    # other lengths through the same graph: the table covers shorter prefixes too
    a.out.fill_(7.0)
    for p, h in zip(a.d_pool, (a.k_pool, a.v_pool)):
        p.copy_(h)
    a.ctx = [300, 0, 0]
    a.start, a.n = [0, 90, 90, 141], [90, 0, 51]
    a.d_idx[1].copy_(i32(a.ctx))
    a.d_idx[2].copy_(i32(a.start))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        with torch.cuda.stream(s1):
            g.replay()
        with torch.cuda.stream(s2):
            b.call()
    a.check()
    b.check()


def test_chunk_captured_behind_copies_and_a_joined_stream(isd):
    """The kernel may start under the one before it: its inputs come from copies,
    a memset and another stream's kernels in the same graph, and it runs twice."""
    c = Chunk(isd, 8, 2, 128, 16, [400, 90, 0], [40, 1, 100], seed=18).upload()
    state = c.d_in + c.d_pool + c.d_idx
    keep = [t.clone() for t in state]
    big = torch.randn(2048, 2048, device="cuda")

    def work():
        main, side = torch.cuda.current_stream(), torch.cuda.Stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            late = (big @ big)[0, 0] * 0
            c.d_pool[0].copy_(keep[3] + late.to(torch.bfloat16))
            c.d_idx[1].copy_(keep[6] + late.int())
        for t, k in list(zip(state, keep))[:3] + [(state[4], keep[4]), (state[7], keep[7])]:
            t.copy_(k)
        c.out.zero_()
        c.out.add_(7.0)
        main.wait_stream(side)
        c.call()
        c.call()

    work()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        work()
    for _ in range(10):
        c.d_in[0].fill_(1.0)
        c.d_idx[1].fill_(3)
        g.replay()
    c.check()


FIRST_CALL = """
import sys, torch
from speculative_verification_isd_b200 import isd
i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
bf = lambda *s: torch.randn(*s, device="cuda", dtype=torch.bfloat16)
d = isd.make_dims(2, 1, 8, 2, 128, 1, 16, 40, 8)
pools, table, kv, used = [bf(40, 16, 2, 128), bf(40, 16, 2, 128)], i32([list(range(8)), list(range(8, 16))]), i32([20, 50]), i32([2, 4])
q, k, v, start, out, ws = bf(9, 8, 128), bf(9, 2, 128), bf(9, 2, 128), i32([0, 4, 9]), bf(9, 1024), isd.alloc_chunk_workspace(d, 9)
new = [i32([0] * 3), i32([0] * 3), torch.empty(3, 8, dtype=torch.int32, device="cuda"), i32([0])]
par, free, moved, live, pws = i32([0, 0, 1]), i32([16]), torch.empty_like(table), i32([0]), isd.alloc_pages_workspace(d)
call = {"chunk": lambda: isd.chunk_attention(d, q, k, v, *pools, table, kv, start, out, ws),
        "fork": lambda: isd.fork_requests(d, par, kv, used, table, free, pools, *new),
        "compact": lambda: isd.compact_pages(d, table, used, pools, moved, live, pws)}[sys.argv[1]]
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    call()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (out, *new, moved, live)]
call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (out, *new, moved, live)))
assert {"chunk": out.isfinite().all(), "fork": new[0].tolist() == [20, 20, 50], "compact": live.item() == 6}[sys.argv[1]]
"""


@pytest.mark.parametrize("what", ["chunk", "fork", "compact"])
def test_first_call_of_a_process_inside_a_capture(what):
    subprocess.run([sys.executable, "-c", FIRST_CALL, what], check=True, timeout=120,
                   cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def test_chunk_call_object_and_larger_workspace(isd):
    c = Chunk(isd, 4, 2, 128, 16, [10], [4], seed=15).upload()
    ws = isd.alloc_chunk_workspace(c.dims, 5000)
    call = isd.ChunkCall(c.dims, *c.d_in, *c.d_pool, *c.d_idx, c.out, ws, c.err)
    for _ in range(3):
        call()
    c.check()


def test_chunk_no_rows(isd):
    c = Chunk(isd, 4, 2, 128, 16, [10, 30], [0, 0], seed=16).upload()
    keep = [p.clone() for p in c.d_pool]
    c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    for p, k in zip(c.d_pool, keep):
        assert torch.equal(p.view(torch.int16), k.view(torch.int16))


@pytest.mark.parametrize("before,after", [(9, 0), (0, 300), (130, 70)])
def test_chunk_rows_of_no_request_only(isd, before, after):
    """Rows, none of them a request's: the kernel runs and writes nothing."""
    c = Chunk(isd, 8, 2, 128, 16, [10, 300, 0], [0, 0, 0], seed=17, before=before, after=after).upload()
    keep = [p.clone() for p in c.d_pool]
    for _ in range(2):
        c.call()
    torch.cuda.synchronize()
    assert int(c.err.item()) == 0
    assert (c.out == 7).all()
    for p, k in zip(c.d_pool, keep):
        assert torch.equal(p.view(torch.int16), k.view(torch.int16))


@pytest.mark.parametrize("P", [16, 20])
def test_far_pages(isd, P):
    """Pages past 2^32 bytes and 2^31 elements of a pool: the same results as in
    a small one, for all three operators."""
    Hq, Hkv, D, cols, far = 8, 2, 128, 20, 5_800_000_000 // (P * 2 * 128 * 2)
    ctx, n = [150, 37, 0], [40, 1, 70]
    used = [-(-(c + m) // P) for c, m in zip(ctx, n)]
    small = 2 * sum(used) + 8
    rng = np.random.default_rng(P)
    q, k, v = bf16(rng, 111, Hq, D).cuda(), bf16(rng, 111, Hkv, D).cuda(), bf16(rng, 111, Hkv, D).cuda()
    data = [bf16(rng, small, P, Hkv, D).cuda() for _ in range(2)]
    ids = rng.permutation(sum(used)) + small // 3
    got = []
    for shift in (0, far - small):
        pages = small + shift
        pools = [torch.empty(pages, P, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        for p, x in zip(pools, data):
            p[shift:] = x
        table = np.full((3, cols), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            table[b, :u] = ids[at:at + u] + shift
            at += u
        d = isd.make_dims(3, 1, Hq, Hkv, D, 1, P, pages, cols)
        out, err = torch.empty(111, Hq * D, dtype=torch.bfloat16, device="cuda"), i32([0])
        isd.chunk_attention(d, q, k, v, *pools, i32(table), i32(ctx), i32(np.cumsum([0] + n)), out,
                            isd.alloc_chunk_workspace(d, 111), err)
        kv, us = i32([c + m for c, m in zip(ctx, n)]), i32(used)
        new = [i32([0] * 2), i32([0] * 2), torch.empty(2, cols, dtype=torch.int32, device="cuda"), i32([0])]
        isd.fork_requests(d, i32([0, 0]), kv, us, i32(table), i32([pages - 4]), pools, *new, err_flag=err)
        tail = [p[new[2][1, new[0][1].item() // P].item(), :new[0][1].item() % P].clone() for p in pools]
        d2 = isd.make_dims(2, 1, Hq, Hkv, D, 1, P, pages, cols)
        isd.compact_pages(d2, new[2], new[1], pools, new[2], new[3], isd.alloc_pages_workspace(d2), err_flag=err)
        rows = [torch.cat([p[j] for j in new[2][r, :new[1][r].item()].tolist()])[:new[0][r].item()]
                for p in pools for r in range(2)]
        assert int(err.item()) == 0
        got.append([out, *tail, *rows, new[3]])
        del pools
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert got[0][-1].item() < small


def test_chunk_rows_past_32_bits(isd):
    """Rows of q and out past 2^32 bytes and 2^31 elements: the last requests'
    rows, and their pages, as by a call of their own."""
    Hq, Hkv, D, P, n, B, last = 32, 8, 128, 16, 120, 4600, 3
    T, per = n * B, -(-n // P)
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(T, h, D, generator=g, device="cuda", dtype=torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pools = [torch.zeros(B * per, P, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table = torch.randperm(B * per, generator=g, device="cuda").to(torch.int32).view(B, per)
    out, err = torch.zeros(T, Hq * D, dtype=torch.bfloat16, device="cuda"), i32([0])
    assert out.numel() > 1 << 31
    d = isd.make_dims(B, 1, Hq, Hkv, D, 1, P, B * per, per)
    isd.chunk_attention(d, q, k, v, *pools, table, i32([0] * B), i32(np.arange(B + 1) * n), out,
                        isd.alloc_chunk_workspace(d, T), err)
    assert int(err.item()) == 0
    rows = slice(T - last * n, T)
    tab = table[-last:].cpu().numpy()
    kp, vp = (O.append(f64(p[table[-last:].long()].flatten(0, 1)) * 0, f64(x[rows]), np.arange(last * per).reshape(last, per),
                       [0] * last, [n * b for b in range(last + 1)]) for p, x in zip(pools, (k, v)))
    for p, want in zip(pools, (kp, vp)):
        assert np.array_equal(f64(p[torch.from_numpy(tab).long().cuda()].flatten(0, 1)), want)
    want = O.chunk_attention(f64(q[rows]), kp, vp, np.arange(last * per).reshape(last, per).tolist(), [0] * last,
                             [n * b for b in range(last + 1)], d.sm_scale)
    check_rows(f64(out[rows]).reshape(last * n, Hq, D), *want, D, n)


def test_chunk_refuses_wrong_tensors(isd):
    c = Chunk(isd, 4, 2, 128, 16, [10], [4], seed=16).upload()
    with pytest.raises(ValueError):
        isd.chunk_attention(c.dims, c.d_in[0].float(), *c.d_in[1:], *c.d_pool, *c.d_idx, c.out, c.ws)
    with pytest.raises(ValueError):
        isd.chunk_attention(c.dims, *c.d_in, *c.d_pool, *c.d_idx, c.out[:2], c.ws)
    with pytest.raises(ValueError):
        isd.chunk_attention(c.dims, c.d_in[0].transpose(1, 2), *c.d_in[1:], *c.d_pool, *c.d_idx, c.out, c.ws)


# ---------------------------------------------------------------- fork
class Cache:
    """A cache of `layers` layers with pages in random order."""

    def __init__(self, isd, B, P, lens, layers=2, Hkv=2, D=64, spare=20, extra=None, cols=None, seed=0):
        rng = np.random.default_rng(seed)
        self.P, self.lens = P, list(lens)
        self.used = [-(-n // P) + (extra[b] if extra else 0) for b, n in enumerate(lens)]
        self.free = sum(self.used)
        self.pages = max(self.free + spare, 1)
        cols = cols or max(max(self.used), 1) + 3
        perm = rng.permutation(max(self.free, 1))
        self.table = np.full((B, cols), -1, np.int32)
        at = 0
        for b, u in enumerate(self.used):
            self.table[b, :u] = perm[at:at + u]
            at += u
        self.dims = isd.make_dims(B, 1, Hkv, Hkv, D, 1, P, self.pages, cols)
        self.pools = [bf16(rng, self.pages, P, Hkv, D).cuda() for _ in range(2 * layers)]
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")


def run_fork(isd, c, parent, reserve=None, free=None, **kw):
    R, cols = len(parent), c.table.shape[1]
    free = c.free if free is None else free
    outs = [torch.full((R,), 99, dtype=torch.int32, device="cuda") for _ in range(2)] + \
        [torch.full((R, cols), 99, dtype=torch.int32, device="cuda"), i32([99])]
    isd.fork_requests(c.dims, i32(parent), i32(c.lens), i32(c.used), i32(c.table), i32([free]), c.pools, *outs,
                      reserve=None if reserve is None else i32(reserve), err_flag=c.err, **kw)
    return outs


def check_fork(isd, c, parent, reserve=None, free=None, flags=0):
    free = c.free if free is None else free
    before = [p.clone() for p in c.pools]
    outs = run_fork(isd, c, parent, reserve, free)
    torch.cuda.synchronize()
    assert int(c.err.item()) == flags
    lens, counts, rows, end, copies = O.fork(parent, reserve or [0] * len(parent), c.lens, c.used, c.table.tolist(),
                                             free, c.pages, c.P)
    assert outs[0].tolist() == lens
    assert outs[1].tolist() == counts
    assert outs[2].tolist() == rows
    assert outs[3].item() == end
    for pool, old in zip(c.pools, before):
        for src, dst, n in copies:
            if 0 <= src < c.pages:
                old[dst, :n] = old[src, :n]
        assert torch.equal(pool, old)


@pytest.mark.parametrize("P", [1, 5, 16, 100])
@pytest.mark.parametrize("parent", [[0, 1, 2], [2, 0, 1], [1, 1, 1, 1], [0], [-1, 2, -1, 2, 0, 2], [-1]])
def test_fork(isd, P, parent):
    lens = [33, 16, 100]
    c = Cache(isd, 3, P, lens, spare=500, extra=[1, 0, 2], cols=140, seed=P)
    check_fork(isd, c, parent)
    check_fork(isd, c, parent, [(7 * i) % 20 for i in range(len(parent))])


def test_fork_many(isd):
    """More requests and slots than a CTA has threads; more pools than a launch takes."""
    B, R = 300, 700
    rng = np.random.default_rng(1)
    c = Cache(isd, B, 4, rng.integers(0, 30, B), layers=70, Hkv=1, D=8, spare=4000, seed=2)
    check_fork(isd, c, rng.integers(-1, B, R).tolist(), rng.integers(0, 9, R).tolist())


def test_fork_as_many_slots_as_go(isd):
    rng = np.random.default_rng(2)
    c = Cache(isd, 2000, 2, rng.integers(0, 9, 2000), layers=1, Hkv=1, D=8, spare=30000, seed=3)
    check_fork(isd, c, rng.integers(-1, 2000, 10000).tolist(), rng.integers(0, 3, 10000).tolist())


def test_fork_faults(isd):
    c = Cache(isd, 3, 16, [33, 16, 100], spare=2, seed=3)
    check_fork(isd, c, [0, 7, -2, 1], flags=isd.FLAG_PARENT_OOB)
    c.err.zero_()
    # two pages are left: the slots that need more come out empty
    check_fork(isd, c, [0, 2, 2, 0, 0, 1], [0, 0, 0, 0, 40, 0], flags=isd.FLAG_CAPACITY)
    c.err.zero_()
    # a list longer than the table; negative room; too few pages for the length
    check_fork(isd, c, [0, 1], [16 * 20, 0], flags=isd.FLAG_CAPACITY)
    c.err.zero_()
    check_fork(isd, c, [0, 1], [-1, 0], flags=isd.FLAG_CAPACITY)
    c.err.zero_()
    c.used[2] = 3
    check_fork(isd, c, [2, 1], flags=isd.FLAG_CAPACITY)


def test_pool_listed_twice(isd):
    """It is copied, and moved, to the same bytes twice."""
    c = Cache(isd, 3, 16, [33, 16, 100], spare=60, extra=[1, 0, 2], cols=20, seed=5)
    c.pools = [c.pools[1], c.pools[0], c.pools[1]]
    check_fork(isd, c, [0, 2, 2, 0])
    c.used[0] = 0
    check_compact(isd, c)


def test_fork_bad_page(isd):
    c = Cache(isd, 2, 16, [40, 20], spare=5, seed=4)
    c.table[0, 2] = 9999
    check_fork(isd, c, [0, 0, 1], flags=isd.FLAG_PAGE_OOB)


# ---------------------------------------------------------------- compact
def check_compact(isd, c, flags=0, in_place=False):
    before = [p.clone() for p in c.pools]
    table = i32(c.table)
    out = table if in_place else torch.full_like(table, 99)
    free = i32([99])
    ws = isd.alloc_pages_workspace(c.dims)
    ws.fill_(0x5A)
    isd.compact_pages(c.dims, table, i32(c.used), c.pools, out, free, ws, err_flag=c.err)
    torch.cuda.synchronize()
    assert int(c.err.item()) == flags
    rows, live, moves = O.compact(c.used, c.table.tolist(), c.pages)
    assert out.tolist() == rows
    assert free.item() == live
    for pool, old in zip(c.pools, before):
        new = old.clone()
        for src, dst in moves:
            new[dst] = old[src]
        assert torch.equal(pool, new)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("used", ["all", "none", "last", "half"])
@pytest.mark.parametrize("P,D", [(1, 8), (5, 64), (16, 128), (100, 64)])
def test_compact(isd, P, D, used, in_place):
    c = Cache(isd, 6, P, [40, 0, 100, 1, 64, 33], D=D, spare=7, seed=P)
    keep = {"all": range(6), "none": [], "last": [5], "half": [1, 2, 4]}[used]
    c.used = [u if b in keep else 0 for b, u in enumerate(c.used)]
    check_compact(isd, c, in_place=in_place)


def test_compact_many_shared_pages(isd):
    """Shared pages move once; more pages than one pass of the planner's block covers."""
    rng = np.random.default_rng(6)
    c = Cache(isd, 200, 1, rng.integers(0, 300, 200), layers=65, Hkv=1, D=8, seed=7)
    for b in range(0, 200, 2):
        n = min(c.used[b], c.used[b + 1])
        c.table[b + 1, :n] = c.table[b, :n]
    c.used = [u if rng.random() < 0.6 else 0 for u in c.used]
    check_compact(isd, c)


@pytest.mark.parametrize("B,cols,pages", [(300, 900, 3000), (4, 20, (1 << 20) + 77)])
def test_compact_large_bookkeeping(isd, B, cols, pages):
    """More table cells, or more pages, than one CTA takes on."""
    rng = np.random.default_rng(9)
    c = Cache(isd, B, 1, rng.integers(0, 9, B), layers=1, Hkv=1, D=8, spare=0, cols=cols, seed=9)
    c.pages = pages
    ids = rng.permutation(pages)[:sum(c.used)]
    at = 0
    for b, u in enumerate(c.used):
        c.table[b, :u] = ids[at:at + u]
        at += u
    c.dims = isd.make_dims(B, 1, 1, 1, 8, 1, 1, pages, cols)
    c.pools = [bf16(rng, pages, 1, 1, 8).cuda() for _ in range(2)]
    c.used = [u if b % 3 else 0 for b, u in enumerate(c.used)]
    check_compact(isd, c)
    c.err.zero_()
    c.table[1, 0] = -7
    c.used[1] = max(c.used[1], 1)
    check_compact(isd, c, flags=isd.FLAG_PAGE_OOB, in_place=True)


def test_compact_faults(isd):
    c = Cache(isd, 3, 16, [33, 16, 100], spare=2, seed=8)
    c.table[0, 1], c.table[2, 0] = 9999, -3
    check_compact(isd, c, flags=isd.FLAG_PAGE_OOB)
    c = Cache(isd, 3, 16, [33, 16, 100], spare=2, seed=9)
    c.used[1] = -4
    check_compact(isd, c, flags=isd.FLAG_CAPACITY)


# ---------------------------------------------------------------- together
def test_prompt_fork_decode_drop_compact(isd):
    """Two prompts go in, one is continued in three ways, every continuation
    decodes on its own tokens, some end, the pages are compacted, and decoding
    goes on: every output is the attention over that answer's own tokens."""
    Hq, Hkv, D, P, cols, pages = 8, 2, 128, 16, 16, 60
    rng = np.random.default_rng(20)
    scale = D ** -0.5
    pools = [torch.full((pages, P, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    err = i32([0])

    def dims(B):
        return isd.make_dims(B, 1, Hq, Hkv, D, 1, P, pages, cols)

    def fork(st, parent, reserve):
        R = len(parent)
        new = [i32([0] * R), i32([0] * R), torch.empty(R, cols, dtype=torch.int32, device="cuda"), i32([0])]
        isd.fork_requests(dims(len(st["hist"])), i32(parent), st["kv"], st["used"], st["table"], st["free"], pools,
                          *new, reserve=i32(reserve), err_flag=err)
        return dict(kv=new[0], used=new[1], table=new[2], free=new[3],
                    hist=[list(st["hist"][p]) if p >= 0 else [] for p in parent])

    def extend(st, n):
        B, T = len(n), sum(n)
        q, k, v = bf16(rng, T, Hq, D), bf16(rng, T, Hkv, D), bf16(rng, T, Hkv, D)
        start = np.concatenate([[0], np.cumsum(n)])
        out = torch.empty(T, Hq * D, dtype=torch.bfloat16, device="cuda")
        d = dims(B)
        isd.chunk_attention(d, q.cuda(), k.cuda(), v.cuda(), *pools, st["table"], st["kv"], i32(start), out,
                            isd.alloc_chunk_workspace(d, T), err)
        st["kv"] = st["kv"] + i32(n)
        got = f64(out).reshape(T, Hq, D)
        for b in range(B):
            st["hist"][b] += [(k[t], v[t]) for t in range(start[b], start[b + 1])]
            m = len(st["hist"][b])
            if n[b] == 0:
                continue
            hk, hv = (torch.stack([h[i] for h in st["hist"][b]])[:, None] for i in (0, 1))
            w = O.chunk_attention(f64(q[start[b]:start[b + 1]]), f64(hk), f64(hv), [list(range(m))], [m - n[b]],
                                  [0, n[b]], scale)
            check_rows(got[start[b]:start[b + 1]], *w, D, m)

    st = dict(kv=i32([0, 0]), used=i32([0, 0]), table=torch.full((2, cols), -1, dtype=torch.int32, device="cuda"),
              free=i32([0]), hist=[[], []])
    st = fork(st, [0, 1], [90, 33])
    extend(st, [90, 33])
    st = fork(st, [0, 1, 0, 0], [7] * 4)
    for _ in range(3):
        extend(st, [1, 1, 1, 1])
    extend(st, [2, 0, 3, 1])
    st = fork(st, [2, -1, 3], [20, 0, 20])
    d = dims(3)
    before = int(st["free"].item())
    isd.compact_pages(d, st["table"], st["used"], pools, st["table"], st["free"], isd.alloc_pages_workspace(d),
                      err_flag=err)
    assert int(st["free"].item()) < before
    extend(st, [5, 0, 17])
    st = fork(st, [2, 0, 0], [30, 30, 30])
    extend(st, [30, 1, 12])
    assert int(err.item()) == 0
