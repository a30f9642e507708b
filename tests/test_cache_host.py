"""Prompt and page operators without a GPU: the oracle's pins and the host-side
refusals of the C ABI and of the Python binding."""
import ctypes
import math

import numpy as np
import pytest

from oracle import cache_oracle as O


@pytest.fixture(scope="module")
def isd():
    from speculative_verification_isd_b200 import build as B
    B.build()
    from speculative_verification_isd_b200 import isd as lib
    return lib


# ------------------------------------------------------------------ oracle
def test_oracle_chunk_attention_is_causal_dense_attention():
    """One request in one page per token against torch's dense attention."""
    import torch
    rng = np.random.default_rng(0)
    kv, n, Hq, Hkv, D = 5, 4, 4, 2, 8
    k, v = rng.normal(size=(2, kv + n, Hkv, D))
    q = rng.normal(size=(n, Hq, D))
    perm = rng.permutation(kv + n)
    pools = []
    for x in (k, v):
        pool = np.zeros((kv + n, 1, Hkv, D))
        pool[perm, 0] = x
        pools.append(pool)
    out, weight, _ = O.chunk_attention(q, *pools, [list(perm)], [kv], [0, n], D ** -0.5)
    tq, tk, tv = (torch.from_numpy(x).transpose(0, 1) for x in (q, k, v))
    mask = torch.ones(n, kv + n).tril(kv).bool()
    ref = torch.nn.functional.scaled_dot_product_attention(
        tq, tk.repeat_interleave(Hq // Hkv, 0), tv.repeat_interleave(Hq // Hkv, 0), mask)
    assert np.allclose(out, ref.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
    assert (weight >= np.abs(out) - 1e-12).all()


def test_oracle_append_touches_only_its_rows():
    pool = np.zeros((4, 3, 1, 2))
    new = np.arange(1, 9, dtype=float).reshape(4, 1, 2)
    got = O.append(pool, new, [[2, 0], [1, 3]], [2, 0], [0, 2, 3])
    want = pool.copy()
    want[2, 2], want[0, 0], want[1, 0] = new[0], new[1], new[2]
    assert np.array_equal(got, want)


def test_oracle_fork_by_hand():
    # request 0: 7 tokens on pages 5, 6 (P = 4) and a spare page 9; request 1: 4 tokens on page 2
    table = [[5, 6, 9, -1], [2, -1, -1, -1]]
    lens, counts, rows, free, copies = O.fork([0, 1, 0, -1, 1], [0, 1, 2, 5, 0], [7, 4], [3, 1], table, 10, 20, 4)
    assert lens == [7, 4, 7, 0, 4] and counts == [3, 2, 3, 0, 1]
    assert rows == [[5, 6, 9, -1], [2, 10, -1, -1], [5, 11, 12, -1], [-1] * 4, [2, -1, -1, -1]]
    assert free == 13 and copies == [(6, 11, 3)]


def test_oracle_compact_by_hand():
    rows, live, moves = O.compact([2, 0, 2], [[7, 1, -1], [3, -1, -1], [5, 7, -1]], 8)
    assert live == 3 and moves == [(5, 0), (7, 2)]
    assert rows == [[2, 1, -1], [-1, -1, -1], [0, 2, -1]]


# ------------------------------------------------------------------ refusals
def _dims(isd, **kw):
    v = dict(B=2, N=1, Hq=4, Hkv=2, D=128, V=1, page_size=16, num_pages=10, max_pages_per_req=4)
    v.update(kw)
    return isd.make_dims(**v)


def test_chunk_refusals(isd):
    lib = isd.library()
    fake = ctypes.c_void_p(1 << 20)   # never dereferenced: validation fails first
    odd = ctypes.c_void_p((1 << 20) + 2)
    d = _dims(isd)
    need = isd.chunk_workspace_bytes(d, 100)
    assert need > 0 and need % 256 == 0
    assert isd.chunk_workspace_bytes(d, -1) == 0
    assert isd.chunk_workspace_bytes(d, 5) <= need

    def call(dd=d, T=100, p=None, ws=fake, n=need):
        return lib.isd_chunk_attention(ctypes.byref(dd), T, *(p or [fake] * 9), ws, n, None, None)

    for i in range(9):
        p = [fake] * 9
        p[i] = None
        assert call(p=p) == isd.ISD_ERR_INVALID_ARG, i
    for i in (0, 1, 2, 3, 4, 8):   # q, k_new, v_new, k_pool, v_pool, out
        p = [fake] * 9
        p[i] = odd
        assert call(p=p) == isd.ISD_ERR_INVALID_ARG, i
    assert call(T=-1) == isd.ISD_ERR_INVALID_ARG
    assert call(ws=None) == isd.ISD_ERR_WORKSPACE
    assert call(n=need - 1) == isd.ISD_ERR_WORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 20) + 16)) == isd.ISD_ERR_WORKSPACE
    big = 1 << 40
    for kw in (dict(D=96), dict(D=256), dict(Hq=258, Hkv=2)):
        assert call(dd=_dims(isd, **kw), n=big) == isd.ISD_ERR_UNSUPPORTED_SHAPE, kw
    for kw in (dict(Hq=3), dict(B=0), dict(page_size=0), dict(num_pages=0), dict(max_pages_per_req=0), dict(D=0)):
        bad = _dims(isd)
        for k, v in kw.items():
            setattr(bad, k, v)
        assert call(dd=bad, n=big) == isd.ISD_ERR_INVALID_ARG, kw
        assert isd.chunk_workspace_bytes(bad, 4) == 0
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(dd=_dims(isd, sm_scale=scale)) == isd.ISD_ERR_INVALID_ARG, scale
    assert lib.isd_chunk_attention(None, 1, *[fake] * 9, fake, need, None, None) == isd.ISD_ERR_INVALID_ARG
    # an output on top of an input (q, k_new, v_new, a pool's last row)
    at = lambda k: ctypes.c_void_p((1 + k) << 24)  # noqa: E731
    for i in (0, 1, 2, 3, 4):
        p = [at(k) for k in range(9)]
        p[8] = ctypes.c_void_p(p[i].value + 16)
        assert call(p=p) == isd.ISD_ERR_INVALID_ARG, i
    p = [at(k) for k in range(9)]
    p[8] = ctypes.c_void_p(p[4].value + d.num_pages * d.page_size * 2 * 128 * 2 - 16)
    assert call(p=p) == isd.ISD_ERR_INVALID_ARG
    for i, j in ((3, 4), (0, 3), (1, 3), (1, 4), (2, 3), (2, 4), (0, 4)):
        p = [at(k) for k in range(9)]
        p[i] = ctypes.c_void_p(p[j].value + 32)
        assert call(p=p) == isd.ISD_ERR_INVALID_ARG, (i, j)
    # no rows: nothing to do, and nothing is launched
    assert call(T=0) == isd.ISD_OK


def test_chunk_refuses_overlaps(isd):
    """What the call writes (out, the pools, the workspace, the flag) overlaps
    nothing else, from the first byte to the last."""
    lib = isd.library()
    d, T = _dims(isd), 100
    need = isd.chunk_workspace_bytes(d, T)
    pool = d.num_pages * d.page_size * d.Hkv * d.D * 2
    # q, k_new, v_new, k_pool, v_pool, page_table, kv_len, q_start, out, ws, err_flag
    size = [T * 4 * 128 * 2, T * 2 * 128 * 2, T * 2 * 128 * 2, pool, pool, 2 * 4 * 4, 2 * 4, 3 * 4, T * 4 * 128 * 2, need, 4]
    align = [16] * 5 + [4] * 3 + [16, 256, 4]
    written = {3, 4, 8, 9, 10}

    def call(p, T=T):
        return lib.isd_chunk_attention(ctypes.byref(d), T, *map(ctypes.c_void_p, p[:9]), ctypes.c_void_p(p[9]), need,
                                       ctypes.c_void_p(p[10]), None)

    for i in range(11):
        for j in range(11):
            if i == j or not {i, j} & written:
                continue
            p = [(1 + k) << 28 for k in range(11)]
            # the last bytes of j under the first of i, as far as i's alignment goes
            p[i] = (p[j] + size[j] - 1) // align[i] * align[i]
            assert call(p) == isd.ISD_ERR_INVALID_ARG, (i, j)
            p[i] = p[j]
            if p[j] % align[i] == 0:
                assert call(p) == isd.ISD_ERR_INVALID_ARG, (i, j)


def test_fork_refusals(isd):
    lib = isd.library()
    at = lambda k: ctypes.c_void_p((1 + k) << 20)  # noqa: E731
    d = _dims(isd)
    pools = (ctypes.c_void_p * 2)(1 << 30, 1 << 31)
    ins, outs = [at(k) for k in range(6)], [at(k + 6) for k in range(4)]

    def call(dd=d, R=3, ins=ins, n=2, pools=pools, outs=outs):
        return lib.isd_fork_requests(ctypes.byref(dd), R, *ins, n, pools, *outs, None, None)

    for i in (0, 2, 3, 4, 5):
        p = list(ins)
        p[i] = None
        assert call(ins=p) == isd.ISD_ERR_INVALID_ARG, i
    for i in range(4):
        p = list(outs)
        p[i] = None
        assert call(outs=p) == isd.ISD_ERR_INVALID_ARG, i
        for j in range(6):   # an output that is an input
            p[i] = ins[j]
            assert call(outs=p) == isd.ISD_ERR_INVALID_ARG, (i, j)
    assert call(R=0) == isd.ISD_ERR_INVALID_ARG
    assert call(n=-1) == isd.ISD_ERR_INVALID_ARG
    assert call(pools=None) == isd.ISD_ERR_INVALID_ARG
    assert call(pools=(ctypes.c_void_p * 2)(1 << 30, None)) == isd.ISD_ERR_INVALID_ARG
    assert call(pools=(ctypes.c_void_p * 2)(1 << 30, (1 << 31) + 8)) == isd.ISD_ERR_INVALID_ARG
    assert call(dd=_dims(isd, B=11998)) == isd.ISD_ERR_UNSUPPORTED_SHAPE
    assert call(R=11999) == isd.ISD_ERR_UNSUPPORTED_SHAPE
    assert call(dd=_dims(isd, Hkv=1, D=4)) == isd.ISD_ERR_UNSUPPORTED_SHAPE
    bad = _dims(isd)
    bad.num_pages = 0
    assert call(dd=bad) == isd.ISD_ERR_INVALID_ARG


def test_fork_refuses_overlaps(isd):
    """Outputs and the flag lie apart from each other and from the inputs, the
    pools from all of them and from each other, to the last byte."""
    lib = isd.library()
    d, R = _dims(isd), 3
    pool = d.num_pages * d.page_size * d.Hkv * d.D * 2
    table = 4 * d.max_pages_per_req
    # parent, reserve, kv_len, pages_used, page_table, next_free_page, the four outputs, err_flag
    size = [12, 12, 8, 8, 2 * table, 4, 12, 12, 3 * table, 4, 4]

    def call(p, pools):
        return lib.isd_fork_requests(ctypes.byref(d), R, *map(ctypes.c_void_p, p[:6]), len(pools),
                                     (ctypes.c_void_p * len(pools))(*pools), *map(ctypes.c_void_p, p[6:]), None)

    apart = [1 << 40, 1 << 41, 1 << 42]
    for i in range(11):
        for j in range(6, 11):
            if i == j:
                continue
            p = [(1 + k) << 20 for k in range(11)]
            for at in (p[j], p[j] + size[j] - 4, p[j] - size[i] + 4):
                p[i] = at
                assert call(p, apart) == isd.ISD_ERR_INVALID_ARG, (i, j)
    for i in range(11):   # a pool's first and last bytes
        for at in (apart[1] - size[i] + 4, apart[1] + pool - 4):
            p = [(1 + k) << 20 for k in range(11)]
            p[i] = at
            assert call(p, apart) == isd.ISD_ERR_INVALID_ARG, i
    p = [(1 + k) << 20 for k in range(11)]
    for pools in ([1 << 40, (1 << 40) + pool - 16], [(1 << 40) + 16, 1 << 41, 1 << 40], [1 << 41, 1 << 40, (1 << 41) - 16]):
        assert call(p, pools) == isd.ISD_ERR_INVALID_ARG


def test_compact_refusals(isd):
    lib = isd.library()
    fake = ctypes.c_void_p(1 << 20)
    d = _dims(isd)
    need = isd.pages_workspace_bytes(d)
    assert need > 0 and need % 256 == 0
    pools = (ctypes.c_void_p * 1)(1 << 30)

    other, free = ctypes.c_void_p(2 << 20), ctypes.c_void_p(3 << 20)

    def call(dd=d, p=(other, fake), n=1, pools=pools, o=(fake, free), ws=fake, k=need):
        return lib.isd_compact_pages(ctypes.byref(dd), *p, n, pools, *o, ws, k, None, None)

    assert call(p=(None, fake)) == isd.ISD_ERR_INVALID_ARG
    assert call(p=(fake, None)) == isd.ISD_ERR_INVALID_ARG
    assert call(o=(None, fake)) == isd.ISD_ERR_INVALID_ARG
    assert call(o=(fake, None)) == isd.ISD_ERR_INVALID_ARG
    assert call(n=-1) == isd.ISD_ERR_INVALID_ARG
    assert call(pools=(ctypes.c_void_p * 1)(None)) == isd.ISD_ERR_INVALID_ARG
    # the new table may be the old one, but not lie across it; nothing else overlaps
    assert call(o=(ctypes.c_void_p((1 << 20) + 4), free)) == isd.ISD_ERR_INVALID_ARG
    assert call(o=(other, free)) == isd.ISD_ERR_INVALID_ARG
    for p in (other, fake, ctypes.c_void_p((1 << 20) + 8)):
        assert call(o=(fake, p)) == isd.ISD_ERR_INVALID_ARG
    assert call(ws=None) == isd.ISD_ERR_WORKSPACE
    assert call(k=need - 1) == isd.ISD_ERR_WORKSPACE
    assert call(ws=ctypes.c_void_p((1 << 20) + 4)) == isd.ISD_ERR_WORKSPACE
    assert call(dd=_dims(isd, Hkv=1, D=4)) == isd.ISD_ERR_UNSUPPORTED_SHAPE
    bad = _dims(isd)
    bad.B = 0
    assert call(dd=bad) == isd.ISD_ERR_INVALID_ARG
    assert isd.pages_workspace_bytes(bad) == 0


@pytest.mark.parametrize("pages", [1, 32, 33, 2 ** 31 - 32, 2 ** 31 - 31, 2 ** 31 - 1])
def test_compact_workspace_of_many_pages(isd, pages):
    """A bit per page in 4-byte words, and three numbers per page and one, each
    part rounded up to 256 bytes."""
    up = lambda n: -(-n // 256) * 256  # noqa: E731
    assert isd.pages_workspace_bytes(_dims(isd, num_pages=pages)) == up(-(-pages // 32) * 4) + up((1 + 3 * pages) * 4)


def test_compact_refuses_overlaps(isd):
    lib = isd.library()
    d = _dims(isd)
    need = isd.pages_workspace_bytes(d)
    pool = d.num_pages * d.page_size * d.Hkv * d.D * 2
    table = 4 * d.B * d.max_pages_per_req
    # pages_used, page_table, next_page_table, next_free_out, ws, err_flag
    size, align = [8, table, table, 4, need, 4], [4, 4, 4, 4, 256, 4]

    def call(p, pools):
        return lib.isd_compact_pages(ctypes.byref(d), *map(ctypes.c_void_p, p[:2]), len(pools),
                                     (ctypes.c_void_p * len(pools))(*pools), *map(ctypes.c_void_p, p[2:5]), need,
                                     ctypes.c_void_p(p[5]), None)

    apart = [1 << 40, 1 << 41, 1 << 42]
    for i in range(6):
        for j in range(2, 6):
            if i == j:
                continue
            p = [(1 + k) << 20 for k in range(6)]
            for at in (p[j], (p[j] + size[j] - 1) // align[i] * align[i]):
                if (i, j, at) == (1, 2, p[2]):
                    continue   # the new table in the old one's place
                p[i] = at
                assert call(p, apart) == isd.ISD_ERR_INVALID_ARG, (i, j)
    for i in range(6):
        p = [(1 + k) << 20 for k in range(6)]
        p[i] = (apart[1] + pool - 1) // align[i] * align[i]
        assert call(p, apart) == isd.ISD_ERR_INVALID_ARG, i
    p = [(1 + k) << 20 for k in range(6)]
    for pools in ([1 << 40, (1 << 40) + pool - 16], [(1 << 40) + 16, 1 << 41, 1 << 40]):
        assert call(p, pools) == isd.ISD_ERR_INVALID_ARG


def test_binding_refuses_host_tensors(isd):
    import torch
    d = _dims(isd)
    z = torch.zeros(8, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        isd.fork_requests(d, z, z, z, z, z, [], z, z, z, z)
    with pytest.raises(ValueError, match="CUDA"):
        isd.compact_pages(d, z, z, [], z, z, z)
    with pytest.raises(ValueError, match="CUDA"):
        isd.chunk_attention(d, *[torch.zeros(0, dtype=torch.bfloat16)] * 5, z, z, z, z, z)
    with pytest.raises(ValueError, match="CUDA"):
        isd.pool_array(d, [torch.zeros(1, dtype=torch.bfloat16)])
    with pytest.raises(ValueError, match="other dims"):
        isd.fork_requests(_dims(isd, num_pages=11), z, z, z, z, z, isd.pool_array(d, []), z, z, z, z)


def test_chunk_call_keeps_the_dims_it_checked(isd, monkeypatch):
    """Dims changed after the check do not reach the kernel with tensors that
    were never compared with them."""
    import torch
    seen = {}

    def pointers(named):
        seen.update((name, n) for name, _, _, n in named)
        return [None] * len(named), 0

    monkeypatch.setattr(isd, "_pointers", pointers)
    d = _dims(isd)
    t = torch.zeros(3 * 4 * 128, dtype=torch.bfloat16)
    call = isd.ChunkCall(d, *[t] * 10, torch.zeros(8, dtype=torch.uint8))
    d.B, d.max_pages_per_req, d.num_pages = 64, 1 << 20, 1 << 20
    kept = call._args[0]._obj
    assert (kept.B, kept.max_pages_per_req, kept.num_pages) == (2, 4, 10)
    assert seen["page_table"] == 8 and seen["q_start"] == 3


def test_rounding_constants():
    """The half steps the GPU tests' tolerances count with."""
    import torch
    assert torch.finfo(torch.bfloat16).eps / 2 == 2.0 ** -8
    assert torch.finfo(torch.float32).eps / 2 == 2.0 ** -24
    assert math.isclose(1.4426950408889634, 1 / math.log(2))
