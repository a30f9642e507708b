"""ISD steps on a cache that the prompt and page operators made.

Prompts go in through isd_chunk_attention, isd_loop runs some steps, the batch
is re-made by isd_fork_requests (one request continued three times, one moved,
one dropped, one slot free for a new request), isd_compact_pages moves its
pages, and isd_loop goes on.  The same steps on a plain batch, in which every
slot has a copy of its cache rows on pages of its own, must give the same bits:
neither the place of a page nor who shares it may show in a result."""
import numpy as np
import pytest
import torch

from speculative_verification_isd_b200 import inputs as I

from gpu_util import bf16_dev, f32_dev, i32_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def isd():
    from speculative_verification_isd_b200 import isd as lib
    return lib


class Model:
    """Weights and tables of a stand-in model, and the buffers of a batch's steps."""

    def __init__(self, isd, D, P, N=4, seed=7):
        self.isd = isd
        self.cfg = I.IsdConfig("cache_loop", B=3, N=N, Hq=8, Hkv=2, D=D, V=1000, page_size=P, prefix_lo=3, prefix_hi=9,
                               w_std=0.4, qkv_std=0.5, kv_std=1.0)
        host = I.make_embedding_tables(self.cfg, seed=seed)
        self.tables = {k: bf16_dev(v) for k, v in host.items()}
        self.W = bf16_dev(I.make_step_inputs(self.cfg, seed=seed, n_clean="one")["W"])
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def dims(self, B, pages, cols):
        c = self.cfg
        return self.isd.make_dims(B, c.N, c.Hq, c.Hkv, c.D, c.V, c.page_size, pages, cols)

    def steps(self, d, pools, state, n_clean, clean_tok, prev_logits, prev_stats, uniforms):
        """isd_loop from a batch's state (kv_len, pages_used, page_table,
        next_free_page), which it updates; returns the batch's other state and
        what the steps emitted."""
        c, B, M, V, n = self.cfg, d.B, d.M, d.V, uniforms.shape[0]
        empty = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        two = lambda t: torch.stack([t, torch.zeros_like(t)])  # noqa: E731
        kv, nc, tok = two(state[0]), two(n_clean), two(clean_tok)
        logits = torch.zeros(2, M * V, dtype=torch.float32, device="cuda")
        stats = torch.zeros(2, M * 4, dtype=torch.int32, device="cuda")
        logits[1], stats[1] = prev_logits.reshape(-1), prev_stats.reshape(-1)
        lens = torch.empty(n, B, dtype=torch.int32, device="cuda")
        toks = torch.empty(n, B, c.N, dtype=torch.int32, device="cuda")
        self.isd.loop(d, n, self.isd.alloc_workspace(d), err_flag=self.err, **self.tables, W=self.W, k_pool=pools[0],
                      v_pool=pools[1], page_table=state[2], pages_used=state[1], next_free_page=state[3], kv_len=kv,
                      n_clean=nc, clean_tok=tok, logits=logits, row_stats=stats, uniforms=f32_dev(uniforms),
                      q=empty(M * c.Hq * c.D), k_new=empty(M * c.Hkv * c.D), v_new=empty(M * c.Hkv * c.D),
                      hidden=empty(M * d.H), accept_len_hist=lens, out_tok_hist=toks)
        last, fin = (n - 1) & 1, n & 1
        state[0] = kv[fin].clone()
        return dict(n_clean=nc[fin].clone(), clean_tok=tok[fin].clone(), logits=logits[last].view(B, -1).clone(),
                    stats=stats[last].view(B, -1).clone(), lens=lens, toks=toks)


def cached_rows(pools, table, kv, P):
    """Of every slot its cached rows in order, K and V."""
    out = []
    for b, n in enumerate(kv.tolist()):
        pos = torch.arange(n, device="cuda")
        page = table[b].long()[pos // P]
        out.append([p[page, pos % P] for p in pools])
    return out


@pytest.mark.parametrize("D,P", [(128, 16), (64, 24)])
def test_loop_on_a_prompted_forked_compacted_cache(isd, D, P):
    m = Model(isd, D, P)
    c, N = m.cfg, m.cfg.N
    pages, cols = 150, 26
    rng = np.random.default_rng(D)
    pools = [torch.full((pages, P, c.Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    normal = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(torch.bfloat16).cuda()  # noqa: E731

    def fork(d, state, parent, reserve):
        R = len(parent)
        new = [i32_dev(np.zeros(R)), i32_dev(np.zeros(R)), torch.empty(R, cols, dtype=torch.int32, device="cuda"),
               i32_dev([0])]
        isd.fork_requests(d, i32_dev(parent), state[0], state[1], state[2], state[3], pools, *new,
                          reserve=i32_dev(reserve), err_flag=m.err)
        return new

    # three prompts, in two pieces
    d = m.dims(3, pages, cols)
    state = [i32_dev([0] * 3), i32_dev([0] * 3), torch.full((3, cols), -1, dtype=torch.int32, device="cuda"), i32_dev([0])]
    state = fork(d, state, [0, 1, 2], [37, 150, 2 * P])
    for n in ([37, 100, P], [0, 50, P]):
        T = sum(n)
        out = torch.empty(T, c.Hq * D, dtype=torch.bfloat16, device="cuda")
        isd.chunk_attention(d, normal(T, c.Hq, D), normal(T, c.Hkv, D), normal(T, c.Hkv, D), *pools, state[2], state[0],
                            i32_dev(np.cumsum([0] + n)), out, isd.alloc_chunk_workspace(d, T), m.err)
        assert torch.isfinite(out).all()
        state[0] = state[0] + i32_dev(n)
    # some steps, each request on its own
    B, MV = 3, d.M * d.V
    tok = torch.full((B, N), -1, dtype=torch.int32)
    tok[:, 0] = torch.from_numpy(rng.integers(0, c.V, B))
    u = lambda seed, n, B: np.stack([I.step_uniforms(seed, k, B, N) for k in range(n)])  # noqa: E731
    first = m.steps(d, pools, state, i32_dev([1] * 3), tok.cuda(), torch.zeros(MV, device="cuda"),
                    torch.zeros(d.M * 4, dtype=torch.int32, device="cuda"), u(1, 5, B))
    assert int(m.err.item()) == 0

    # request 1 goes on three times, request 0 in another slot, request 2 ends, slot 2 is free
    parent = [1, 0, -1, 1, 1]
    R = len(parent)
    new = fork(d, state, parent, [0, 3, 0, 40, 0])
    d = m.dims(R, pages, cols)
    free = int(new[3].item())
    isd.compact_pages(d, new[2], new[1], pools, new[2], new[3], isd.alloc_pages_workspace(d), err_flag=m.err)
    assert int(m.err.item()) == 0
    assert int(new[3].item()) < free
    # the rest of a request's state follows by the same parents; a new request begins in slot 2
    at = torch.tensor([max(p, 0) for p in parent], device="cuda")
    rest = {k: first[k][at].clone() for k in ("n_clean", "clean_tok", "logits", "stats")}
    rest["n_clean"][2], rest["clean_tok"][2, 0], rest["clean_tok"][2, 1:] = 1, 5, -1

    # the plain batch: copies of every slot's rows on pages of its own
    kv = new[0].clone()
    rows = cached_rows(pools, new[2], kv, P)
    plain_pools = [torch.full((R * cols, P, c.Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    plain_table = torch.full((R, cols), -1, dtype=torch.int32, device="cuda")
    used, nxt = [], 0
    for b, n in enumerate(kv.tolist()):
        used.append(-(-n // P))
        ids = torch.arange(nxt, nxt + used[b], device="cuda")
        plain_table[b, :used[b]] = ids.to(torch.int32)
        pos = torch.arange(n, device="cuda")
        for pool, x in zip(plain_pools, rows[b]):
            pool[ids[pos // P], pos % P] = x
        nxt += used[b]
    plain = [kv, i32_dev(used), plain_table, i32_dev([nxt])]

    steps = 7
    got = m.steps(d, pools, new, rest["n_clean"], rest["clean_tok"], rest["logits"], rest["stats"], u(2, steps, R))
    d_plain = m.dims(R, R * cols, cols)
    want = m.steps(d_plain, plain_pools, plain, rest["n_clean"], rest["clean_tok"], rest["logits"], rest["stats"],
                   u(2, steps, R))
    assert int(m.err.item()) == 0
    for k in want:
        assert torch.equal(got[k], want[k]), k
    assert torch.equal(new[0], plain[0])
    assert torch.isfinite(got["logits"]).all()
    # the three continuations drew their own uniforms: they are three answers now
    assert len({tuple(got["toks"][:, b].flatten().tolist()) for b in (0, 3, 4)}) == 3
    for x, y in zip(cached_rows(pools, new[2], new[0], P), cached_rows(plain_pools, plain[2], plain[0], P)):
        for a, b in zip(x, y):
            assert torch.equal(a, b) and torch.isfinite(a).all()
