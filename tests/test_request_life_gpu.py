"""A request's life through the C ABI: rows reserved, prompts appended and
attended over, one continuation forked, a token tree verified with its log
probabilities, the path committed and its pages released, the fork freed, the
pool compacted, and single tokens attended over what is left."""
import math

import numpy as np
import pytest
import torch

import workloads as W
import tree_speculative_verification_spec_gb300 as S
from request_life import logprob_reference, prompt_reference
from tree_speculative_verification_spec_gb300.pipeline import DeviceBatch, PromptPass, VerifyPass

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Pool:
    """Two layers of caches, a block table and a pool; every slot starts as NaN."""

    def __init__(self, rows, max_blocks, num_blocks, Hkv, bs, D, layers=2):
        self.shape = (rows, max_blocks, bs, num_blocks)
        self.caches = [[torch.full((num_blocks, Hkv, bs, D), math.nan, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
                       for _ in range(layers)]
        self.k, self.v = (torch.tensor([c[i].data_ptr() for c in self.caches], dtype=torch.int64, device="cuda") for i in (0, 1))
        self.layers, self.Hkv, self.D = layers, Hkv, D
        self.table = torch.full((rows, max_blocks), -1, dtype=torch.int32, device="cuda")
        perm = torch.randperm(num_blocks, generator=torch.Generator().manual_seed(1)).to(torch.int32)
        self.pool, self.count = perm.cuda(), _ints([num_blocks])
        self.ws = torch.empty(S.spec_pages_workspace_size(rows, max_blocks, num_blocks, rows), dtype=torch.uint8, device="cuda")

    def fork(self, src, dst, length, room):
        st = _ints([77] * len(src))
        S.spec_pages_fork(self.k, self.v, self.layers, self.table, *self.shape, _ints(src), _ints(dst), _ints(length), _ints(room),
                          len(src), self.Hkv, self.D, S.SPEC_BF16, self.pool, self.count, self.ws, st)
        assert st.tolist() == [0] * len(src)

    def free(self, rows):
        st = _ints([77] * len(rows))
        S.spec_pages_free(self.table, *self.shape, _ints(rows), None, len(rows), self.pool, self.count, self.ws, st)
        assert st.tolist() == [0] * len(rows)

    def compact(self):
        st, moved, page_map = _ints([77]), _ints([77]), _ints([0] * self.shape[3])
        S.spec_pages_compact(self.k, self.v, self.layers, self.table, *self.shape, self.Hkv, self.D, S.SPEC_BF16, self.pool, self.count,
                             page_map, moved, self.ws, st)
        assert st.tolist() == [0]
        return moved.item()

    def held(self):
        return len({p for p in self.table.flatten().tolist() if p >= 0})


def _attend(pool, rows, q, lens, prefix, kv=None, layer=0):
    """PromptPass over the given table rows, held to 64-bit attention over the cache."""
    k, v = pool.caches[layer]
    off = _ints(np.concatenate([[0], np.cumsum(lens)]).tolist())
    table = pool.table[torch.tensor(rows, device="cuda")].contiguous()
    p = PromptPass(q, k, v, table, off, _ints(prefix), max(lens), max(prefix), 1.0 / math.sqrt(pool.D))
    p.run(kv)
    assert p.status.tolist() == [0] * len(rows)
    d = dict(q=q, k=k, v=v, table=table, seq_off=off, prefix=_ints(prefix), B=len(rows), T=q.shape[0], Hq=q.shape[1], Hkv=pool.Hkv,
             D=pool.D, bs=pool.shape[2], scale=1.0 / math.sqrt(pool.D))
    ref, tol = prompt_reference(d)
    assert ((p.out.double() - ref).abs() <= tol).all()
    return p.out


def test_a_request_from_its_prompt_to_its_answer():
    g = torch.Generator("cuda").manual_seed(5)
    Hq, Hkv, D, bs, V = 8, 2, 64, 16, 700
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    pool = Pool(rows=4, max_blocks=96, num_blocks=300, Hkv=Hkv, bs=bs, D=D)
    lens = [1203, 37]
    # ---- rows for both prompts; the prompts in two chunks, every layer
    pool.fork([-1, -1], [0, 1], [0, 0], [lens[0], lens[1]])
    cut = [700, 0]
    for layer in range(2):
        for a, n, prefix in ((0, cut, [0, 0]), (1, [lens[0] - cut[0], lens[1]], [cut[0], 0])):
            T = sum(n)
            _attend(pool, [0, 1], rand(T, Hq, D), n, prefix, (rand(T, Hkv, D), rand(T, Hkv, D)), layer)
    before = [[c.clone() for c in pair] for pair in pool.caches]
    # ---- request 0 goes on in a second row, and every row gets room for its tree
    pool.fork([0], [2], [lens[0]], [0])
    shared = lens[0] // bs
    assert torch.equal(pool.table[0, :shared], pool.table[2, :shared]) and pool.table[0, shared] != pool.table[2, shared]
    for pair, old in zip(pool.caches, before):
        for c, o in zip(pair, old):
            tail = lens[0] % bs
            assert torch.equal(c[pool.table[2, shared], :, :tail], o[pool.table[0, shared], :, :tail])
    held = [lens[0], lens[1], lens[0]]
    trees = [12, 5, 20]
    pool.fork([0, 1, 2], [0, 1, 2], held, trees)
    before_pass = pool.count.item()
    # ---- one verification pass over three trees, with log probabilities
    rng = np.random.default_rng(9)
    parent = np.concatenate([[-1] + [int(rng.integers(0, i)) for i in range(1, n)] for n in trees]).astype(np.int32)
    off = np.concatenate([[0], np.cumsum(trees)]).astype(np.int32)
    T = int(off[-1])
    logits = rng.standard_normal((T, V)).astype(np.float32) * 2
    tokens = rng.permutation(V)[:T].astype(np.int32)
    for b in range(3):  # the greedy walk goes down some edges
        for u in range(1, trees[b]):
            if rng.random() < 0.7:
                p = int(parent[off[b] + u])
                logits[off[b] + p, tokens[off[b] + u]] = 9.0 + rng.random()
    k, v = pool.caches[0]
    batch = DeviceBatch(B=3, T=T, n_max=max(trees), V=V, Hq=Hq, Hkv=Hkv, D=D, block_size=bs, num_blocks=300, max_prefix=max(held),
                        parent=_ints(parent.tolist()), tree_off=_ints(off.tolist()), tokens=_ints(tokens.tolist()),
                        prefix_len=_ints(held), block_table=pool.table[:3].contiguous(), q=rand(T, Hq, D), k_cache=k, v_cache=v,
                        p_logits=torch.from_numpy(logits).cuda(), q_probs=None, uniforms=None, scale=1.0 / math.sqrt(D))
    vp = VerifyPass(batch, logprob_top=4)
    vp.run("greedy", commit=False, tree_kv=(rand(T, Hkv, D), rand(T, Hkv, D)))
    assert vp.status.tolist() == [0, 0, 0]
    path, alen, emitted = vp.path.tolist(), vp.accept_len.tolist(), vp.emitted.tolist()
    assert max(alen) > 1
    for b in range(3):
        for i in range(max(trees)):
            if i >= alen[b]:
                assert math.isnan(vp.logprob[b, i].item()) and vp.rank[b, i].item() == -1
                continue
            lp, ent, rank, top, top_lp = logprob_reference(logits[off[b] + path[b][i]], emitted[b][i], 1.0, 4)
            assert vp.rank[b, i].item() == rank == 0  # greedy: the most likely token
            assert abs(vp.logprob[b, i].item() - lp) < 1e-4 and abs(vp.entropy[b, i].item() - ent) < 1e-4
            assert vp.top_tokens[b, i].tolist() == list(top)
            assert np.abs(vp.top_logprobs[b, i].cpu().numpy() - top_lp).max() < 1e-4
    # ---- the path stays, the tree's other pages go back
    new_len = torch.zeros(3, dtype=torch.int32, device="cuda")
    table = batch.block_table
    S.spec_kv_commit_layers(pool.k, pool.v, 2, table, 96, bs, 300, batch.prefix_len, batch.tree_off, vp.path, batch.n_max,
                            vp.accept_len, 3, Hkv, D, S.SPEC_BF16, new_len, pool.pool, pool.count, vp.status)
    assert vp.status.tolist() == [0, 0, 0]
    pool.table[:3] = table
    assert new_len.tolist() == [h + a for h, a in zip(held, alen)]
    assert pool.count.item() >= before_pass and pool.count.item() + pool.held() == 300
    # ---- the fork ends; what is left comes together; single tokens go on over it
    q1 = rand(2, Hq, D)
    lens_now = new_len.tolist()
    # layer 0 holds the accepted tokens' K/V: the last one attends to all before it
    first = _attend(pool, [0, 1], q1, [1, 1], [n - 1 for n in lens_now[:2]])
    pool.free([2])
    assert pool.count.item() + pool.held() == 300
    moved = pool.compact()
    assert moved > 0 and max(pool.table.flatten().tolist()) == pool.held() - 1
    again = _attend(pool, [0, 1], q1, [1, 1], [n - 1 for n in lens_now[:2]])
    assert torch.equal(first, again)
    pool.free([0, 1])
    assert pool.count.item() == 300 and sorted(pool.pool.tolist()) == list(range(300))


def test_logprobs_need_their_buffers():
    w = W.small_random(3, B=1, n_range=(4, 4), V=50)
    with pytest.raises(ValueError):
        VerifyPass(DeviceBatch.from_workload(w)).logprobs()


def test_temperatures_that_only_the_log_probabilities_refuse():
    """The verifiers take what the log probabilities flag (a greedy pass ignores
    temperatures, a stochastic one takes any above 0): the accepted path is
    committed all the same, and the flag stands in a word of its own."""
    for mode, temps, bad in (("greedy", [0.0, 1.0, math.inf], [0, 2]), ("stochastic", [1e-31, 1.0, 2.0], [0])):
        w = W.small_random(11, B=3, n_range=(6, 9), V=60)
        plain = VerifyPass(DeviceBatch.from_workload(w))
        plain.inv_temp = None if mode == "greedy" else torch.tensor(temps, device="cuda")
        plain.run(mode)
        b = DeviceBatch.from_workload(w)
        vp = VerifyPass(b, logprob_top=2)
        vp.inv_temp = torch.tensor(temps, device="cuda")
        vp.run(mode)
        assert plain.status.tolist() == vp.status.tolist() == [0, 0, 0]
        assert vp.accept_len.tolist() == plain.accept_len.tolist() and vp.new_len.tolist() == plain.new_len.tolist()
        assert vp.new_len.tolist() == [p + a for p, a in zip(b.prefix_len.tolist(), vp.accept_len.tolist())]
        for x, y in ((plain.batch.k_cache, b.k_cache), (plain.batch.v_cache, b.v_cache)):
            assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                               y.view(torch.int16 if y.dtype == torch.bfloat16 else torch.int32))
        assert vp.logprob_status.tolist() == [S.SPEC_DEV_BAD_TEMP if r in bad else 0 for r in range(3)]
        for r in range(3):
            assert all(math.isnan(v) == (r in bad) for v in vp.logprob[r, :vp.accept_len[r]].tolist())
        vp.inv_temp = torch.ones(3, device="cuda")   # the word is the last pass's
        vp.mask_build()
        vp.verify(mode)
        vp.logprobs()
        assert vp.logprob_status.tolist() == [0, 0, 0]


def test_a_prompt_pass_runs_again_after_a_refusal():
    """A request that one run flagged is computed by the next, on the pass's own
    stream too."""
    g = torch.Generator("cuda").manual_seed(21)
    Hq, Hkv, D, bs, n = 4, 2, 64, 16, 50
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    k, v = (torch.zeros((16, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8).contiguous()
    q, kv = rand(2 * n, Hq, D), (rand(2 * n, Hkv, D), rand(2 * n, Hkv, D))
    for stream in (None, torch.cuda.Stream()):
        prefix = _ints([10, 41])
        p = PromptPass(q, k, v, table, _ints([0, n, 2 * n]), prefix, n, 40, 1.0 / math.sqrt(D))
        p.out.fill_(7.0)
        torch.cuda.synchronize()
        p.run(kv, stream=stream)
        torch.cuda.synchronize()
        assert p.status.tolist() == [0, S.SPEC_DEV_CAPACITY] and (p.out[n:] == 7.0).all()
        prefix[1] = 0
        torch.cuda.synchronize()
        p.run(kv, stream=stream)
        torch.cuda.synchronize()
        assert p.status.tolist() == [0, 0]
        d = dict(q=q, k=k, v=v, table=table, seq_off=_ints([0, n, 2 * n]), prefix=prefix, B=2, T=2 * n, Hq=Hq, Hkv=Hkv, D=D, bs=bs,
                 scale=1.0 / math.sqrt(D))
        ref, tol = prompt_reference(d)
        assert ((p.out.double() - ref).abs() <= tol).all()


def test_a_prompt_right_behind_the_kernels_that_make_its_rows():
    """Rows, pages and lengths written by the kernels just before the pass, a
    library product among them, as a model's layers do."""
    g = torch.Generator("cuda").manual_seed(31)
    Hq, Hkv, D, bs, n, width = 8, 2, 128, 16, 2048, 512
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    x, wk, wv, wq = rand(2 * n, width), rand(width, Hkv * D), rand(width, Hkv * D), rand(width, Hq * D)
    want = None
    for turn in range(6):
        pool = Pool(rows=2, max_blocks=n // bs + 1, num_blocks=300, Hkv=Hkv, bs=bs, D=D, layers=1)
        src, dst, zero, room = _ints([-1, -1]), _ints([0, 1]), _ints([0, 0]), _ints([n, n])
        off, prefix, st = _ints([0, n, 2 * n]), _ints([0, 0]), _ints([7, 7])
        p = PromptPass(rand(2 * n, Hq, D), *pool.caches[0], pool.table, off, prefix, n, 0, 0.01)
        torch.cuda.synchronize()
        p.q = (x @ wq).view(2 * n, Hq, D)
        S.spec_pages_fork(None, None, 0, pool.table, *pool.shape, src, dst, zero, room, 2, Hkv, D, S.SPEC_BF16, pool.pool, pool.count, pool.ws, st)
        k, v = (x @ wk).view(2 * n, Hkv, D), (x @ wv).view(2 * n, Hkv, D)
        p.run((k, v))
        assert p.status.tolist() == [0, 0] and st.tolist() == [0, 0]
        got = [c[pool.table[b, :n // bs].long()].transpose(1, 2).reshape(n, Hkv, D) for c in pool.caches[0] for b in (0, 1)]
        assert torch.equal(torch.cat(got[:2]), k) and torch.equal(torch.cat(got[2:]), v)
        want = p.out.clone() if want is None else want
        assert torch.equal(p.out, want)


@pytest.mark.parametrize("dtype,D,bs", [(torch.bfloat16, 128, 16), (torch.float32, 64, 256), (torch.bfloat16, 64, 8)])
def test_append_of_more_rows_than_a_tree_has(dtype, D, bs):
    """Prompts of thousands of rows beside short, empty and refused ones: the
    caches byte for byte."""
    g = torch.Generator().manual_seed(bs)
    Hkv = 3
    lens, prefix = [5000, 0, 1, 1025, 300, 40], [37, 9, 4095, 0, 90, 17]
    used = [-(-(n + p) // bs) for n, p in zip(lens, prefix)]
    nb, width = sum(used) + 5, max(used)
    perm = torch.randperm(nb, generator=g).tolist()
    table = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = torch.tensor(perm[at:at + u], dtype=torch.int32)
        at += u
    table[4, used[4] - 1] = nb                       # a bad id among the pages to be written
    prefix[5] = width * bs - 39                      # one slot short
    off = [0] + np.cumsum(lens).tolist()
    bits = torch.int16 if dtype == torch.bfloat16 else torch.int32
    make = lambda *s: torch.randint(0, 1 << 14, s, generator=g, dtype=torch.int32).to(bits)  # noqa: E731
    new = [make(off[-1], Hkv, D) for _ in range(2)]
    caches = [make(nb, Hkv, bs, D) for _ in range(2)]
    dev = [c.cuda().view(dtype) for c in caches]
    status = _ints([0] * len(lens))
    S.spec_kv_append(*[n.cuda().view(dtype) for n in new], *dev, table.cuda(), width, bs, nb, _ints(prefix), _ints(off), len(lens),
                     max(lens), Hkv, D, status)
    assert status.tolist() == [0, 0, 0, 0, S.SPEC_DEV_BAD_BLOCK, S.SPEC_DEV_CAPACITY]
    for c, n in zip(caches, new):
        for b in range(4):
            s = prefix[b] + torch.arange(lens[b])
            c[table[b][s // bs].long(), :, s % bs] = n[off[b]:off[b + 1]]
    for c, d in zip(caches, dev):
        assert torch.equal(c, d.cpu().view(bits))


def test_page_calls_take_cache_addresses_of_64_bits_alone():
    pool = Pool(rows=2, max_blocks=4, num_blocks=8, Hkv=1, bs=8, D=64)
    one, st = _ints([0]), _ints([77])
    for k, v in ((pool.k.int(), pool.v), (pool.k, pool.v.float()), (pool.k[:1], pool.v), (None, pool.v)):
        with pytest.raises((ValueError, S.SpecError)):
            S.spec_pages_fork(k, v, pool.layers, pool.table, *pool.shape, _ints([-1]), one, one, _ints([5]), 1, 1, 64, S.SPEC_BF16,
                              pool.pool, pool.count, pool.ws, st)
        with pytest.raises((ValueError, S.SpecError)):
            S.spec_pages_compact(k, v, pool.layers, pool.table, *pool.shape, 1, 64, S.SPEC_BF16, pool.pool, pool.count,
                                 torch.zeros(8, dtype=torch.int32, device="cuda"), one, pool.ws, st)
    assert st.tolist() == [77] and pool.count.item() == 8


def test_a_captured_prompt_pass():
    """A pass replayed from a graph: the status it clears, the rows it appends and
    the lengths as they are at each replay."""
    g = torch.Generator("cuda").manual_seed(41)
    Hq, Hkv, D, bs, n = 4, 2, 64, 16, 60
    rand = lambda *s: torch.randn(s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    k, v = (torch.zeros((24, Hkv, bs, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(2, 12).contiguous()
    q, kv = rand(2 * n, Hq, D), (rand(2 * n, Hkv, D), rand(2 * n, Hkv, D))
    prefix = _ints([0, 90])
    p = PromptPass(q, k, v, table, _ints([0, n, 2 * n]), prefix, n, 90, 1.0 / math.sqrt(D))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        p.run(kv)
    for length, flag in ((90, 0), (91, S.SPEC_DEV_CAPACITY), (64, 0)):
        prefix[1] = length
        for t in (q, *kv):
            t.copy_(rand(*t.shape))
        graph.replay()
        torch.cuda.synchronize()
        assert p.status.tolist() == [0, flag]
        sound = 2 if flag == 0 else 1
        d = dict(q=q, k=k, v=v, table=table, seq_off=_ints([0, n, 2 * n]), prefix=prefix, B=sound, T=2 * n, Hq=Hq, Hkv=Hkv, D=D, bs=bs,
                 scale=1.0 / math.sqrt(D))
        ref, tol = prompt_reference(d)
        assert ((p.out.double() - ref).abs() <= tol)[:sound * n].all()
