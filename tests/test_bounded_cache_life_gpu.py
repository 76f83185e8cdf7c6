"""A request on a budget through the pipeline: prompts projected, rotated and
attended over, their slots weighed, every row cut to a budget and its old pages
freed, then token trees projected at the positions of the whole text, verified
over the short rows, committed and weighed again."""
import math

import numpy as np
import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from bounded_cache import ints, keep_reference, offsets, rope_reference, weight_reference
from request_life import prompt_reference
from test_request_life_gpu import Pool
from tree_speculative_verification_spec_gb300.pipeline import CacheBudget, DeviceBatch, PromptPass, Rotary, VerifyPass

pytestmark = pytest.mark.gpu
Hq, Hkv, D, BS, LAYERS, V = 8, 2, 64, 16, 2, 97


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


def _projection(T, seed):
    return torch.randn((T, Hq + 2 * Hkv, D), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def _rows(cache, table, row, h, n):
    """The first n slots of kv-head h of a table row."""
    return cache[table[row, :-(-n // BS)].long(), h].reshape(-1, D)[:n]


def _weights_hold(budget, layer, row, before, d, **kw):
    ref, tol = weight_reference(d, before, budget.decay, **kw)
    got = budget.weight[layer, row:row + len(d["prefix"])]
    mine = ~ref.isnan()
    assert ((got.double() - ref).abs()[mine] <= tol[mine]).all()


def test_prompts_budget_trees():
    lens, keep, first, last = [300, 170], [64, 50], 4, 16
    pool = Pool(4, 24, 80, Hkv, BS, D, LAYERS)
    k_of, v_of = [c[0] for c in pool.caches], [c[1] for c in pool.caches]
    g = torch.Generator().manual_seed(2)
    freq = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    norm = [(1 + 0.2 * torch.randn(D, generator=g)).bfloat16().cuda() for _ in range(2)]
    rotary = Rotary(freq, D, q_norm=norm[0], k_norm=norm[1], eps=1e-5)
    budget = CacheBudget(LAYERS, 4, Hkv, 24 * BS, decay=0.5)
    off, zero, scale = offsets(lens), ints([0, 0]), 1 / math.sqrt(D)

    # prompts into rows 0 and 1
    pool.fork([-1, -1], [0, 1], [0, 0], lens)
    for layer in range(LAYERS):
        qkv = _projection(sum(lens), 10 + layer)
        q = torch.empty((sum(lens), Hq, D), dtype=torch.bfloat16, device="cuda")
        p = PromptPass(q, k_of[layer], v_of[layer], pool.table[:2], off, zero, max(lens), 0, scale)
        p.run(prompt_qkv=qkv, rotary=rotary)
        budget.observe_prompt(layer, p, window=32)
        assert p.status.tolist() == [0, 0]
        place = torch.cat([torch.arange(n) for n in lens]).cuda()[:, None].expand(-1, D // 2)
        ref, tol = rope_reference(qkv, Hq, Hkv, D, 0, freq, place, *norm, 1e-5)
        assert ((q.double() - ref[:, :Hq]).abs() <= tol[:, :Hq]).all()
        at = off.tolist()
        for b in range(2):
            for h in range(Hkv):
                got = _rows(k_of[layer], pool.table, b, h, lens[b])
                assert ((got.double() - ref[at[b]:at[b + 1], Hq + h]).abs() <= tol[at[b]:at[b + 1], Hq + h]).all()
                assert torch.equal(_rows(v_of[layer], pool.table, b, h, lens[b]), qkv[at[b]:at[b + 1], Hq + Hkv + h])
        d = dict(q=q, k=k_of[layer], v=v_of[layer], table=pool.table[:2], seq_off=off, prefix=zero, B=2, T=sum(lens), Hq=Hq, Hkv=Hkv, D=D, bs=BS, scale=scale,
                 stride=24 * BS)
        out, tol = prompt_reference(d)
        assert ((p.out.double() - out).abs() <= tol).all()
        _weights_hold(budget, layer, 0, None, d, window=32)

    # cut to rows 2 and 3 (with room for a tree), old rows freed
    nodes = [7, 5]
    pool.fork([-1, -1], [2, 3], [0, 0], [k + n for k, n in zip(keep, nodes)])
    held = [[[_rows(c[i], pool.table, b, h, lens[b]).clone() for i in range(2)] for b in range(2) for h in range(Hkv)] for c in pool.caches]
    old = budget.weight.clone()
    slots, new_len, st = budget.evict(pool.k, pool.v, pool.table, BS, 80, ints([0, 1]), ints([2, 3]), ints(lens), max(keep), first, last, D, S.SPEC_BF16,
                                      keep=ints(keep))
    pool.free([0, 1])
    assert new_len.tolist() == keep and st.tolist() == [0, 0]
    for layer in range(LAYERS):
        for b in range(2):
            for h in range(Hkv):
                stay = keep_reference(old[layer, b, h].tolist(), lens[b], keep[b], first, last)
                assert slots[layer, b, h, :keep[b]].tolist() == stay
                assert torch.equal(budget.weight[layer, 2 + b, h, :keep[b]], old[layer, b, h, torch.tensor(stay, device="cuda")])
                for i in range(2):
                    got = _rows(pool.caches[layer][i], pool.table, 2 + b, h, keep[b])
                    assert torch.equal(got, held[layer][b * Hkv + h][i][torch.tensor(stay, device="cuda")])

    # token trees at the positions behind the whole text, over the short rows
    parent = [[-1, 0, 0, 1, 3, 2, 4], [-1, 0, 1, 2, 0]]
    tree_off, T = offsets(nodes), sum(nodes)
    greedy = torch.randint(0, V, (T,), generator=g)
    logits = torch.randn((T, V), generator=g)
    logits[torch.arange(T), greedy] += 20
    tokens = torch.randint(0, V, (T,), generator=g)
    for b, path in enumerate(([1, 3, 4], [1, 2])):  # what a greedy walk accepts
        at = int(tree_off[b])
        for c in path:
            tokens[at + c] = greedy[at + parent[b][c]]
    base, prefix = ints(lens), ints(keep)
    for layer in range(LAYERS):
        qkv = _projection(T, 20 + layer)
        batch = DeviceBatch(B=2, T=T, n_max=max(nodes), V=V, Hq=Hq, Hkv=Hkv, D=D, block_size=BS, num_blocks=80, max_prefix=max(keep),
                            parent=ints(sum(parent, [])), tree_off=tree_off, tokens=tokens.to(torch.int32).cuda(), prefix_len=prefix, block_table=pool.table[2:],
                            q=torch.empty((T, Hq, D), dtype=torch.bfloat16, device="cuda"), k_cache=k_of[layer], v_cache=v_of[layer], p_logits=logits.cuda(),
                            q_probs=None, uniforms=None, scale=scale)
        v = VerifyPass(batch)
        v.run("greedy", commit=False, tree_qkv=qkv, rotary=rotary, pos_base=base)
        assert v.status.tolist() == [0, 0]
        depth = []
        for par in parent:
            own = []
            for x in par:
                own.append(0 if x < 0 else own[x] + 1)
            depth.append(own)
        place = torch.tensor([n + x for n, own in zip(lens, depth) for x in own], device="cuda")[:, None].expand(-1, D // 2)
        ref, tol = rope_reference(qkv, Hq, Hkv, D, 0, freq, place, *norm, 1e-5)
        assert ((batch.q.double() - ref[:, :Hq]).abs() <= tol[:, :Hq]).all()
        tree_k = [[_rows(k_of[layer], pool.table, 2 + b, h, keep[b] + nodes[b])[keep[b]:].clone() for h in range(Hkv)] for b in range(2)]
        for b in range(2):
            a0, a1 = int(tree_off[b]), int(tree_off[b + 1])
            for h in range(Hkv):
                assert ((tree_k[b][h].double() - ref[a0:a1, Hq + h]).abs() <= tol[a0:a1, Hq + h]).all()
                # attention of every node over the kept slots and its ancestors
                k = _rows(k_of[layer], pool.table, 2 + b, h, keep[b] + nodes[b]).double()
                vv = _rows(v_of[layer], pool.table, 2 + b, h, keep[b] + nodes[b]).double()
                for u in range(nodes[b]):
                    up, x = [], u
                    while x >= 0:
                        up.append(keep[b] + x)
                        x = parent[b][x]
                    see = torch.tensor(list(range(keep[b])) + up, device="cuda")
                    q = batch.q[a0 + u, h * 4:h * 4 + 4].double()
                    w = torch.softmax(q @ k[see].T * scale, -1)
                    want, size = w @ vv[see], w @ vv[see].abs()
                    err = (v.out[a0 + u, h * 4:h * 4 + 4].double() - want).abs()
                    # half a step on the output, on every weight and on their sum; 1e-4 for 32 bits
                    assert (err <= 2.0 ** -8 * (want.abs() + 2 * size) + 1e-4 * size).all()
        v.commit()
        budget.observe_path(layer, v, row=2)
        assert v.accept_len.tolist() == [4, 3] and v.new_len.tolist() == [keep[0] + 4, keep[1] + 3] and v.status.tolist() == [0, 0]
        d = dict(q=batch.q, k=k_of[layer], table=pool.table[2:], seq_off=tree_off, prefix=prefix, Hq=Hq, Hkv=Hkv, D=D, bs=BS, scale=scale)
        before = torch.stack([old[layer, b, :, :] for b in range(2)])
        for b in range(2):
            for h in range(Hkv):
                before[b, h, :keep[b]] = old[layer, b, h, slots[layer, b, h, :keep[b]].long()]
        _weights_hold(budget, layer, 2, before, d, path=np.array([[0, 1, 3, 4], [0, 1, 2, -1]]), accept=[4, 3])


def test_budget_refuses_what_is_not_its_own():
    budget = CacheBudget(1, 2, Hkv, 64)
    q, k = torch.zeros((3, Hq, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((4, Hkv, BS, D), dtype=torch.bfloat16, device="cuda")
    p = PromptPass(q, k, k, ints([[0]]), ints([0, 3]), ints([0]), 3, 0, 0.1)
    for kw in (dict(layer=1), dict(layer=0, row=2), dict(layer=-1)):
        with pytest.raises(ValueError):
            budget.observe_prompt(kw.pop("layer"), p, **kw)


def test_budget_on_a_stream_of_its_own():
    """Observed and evicted on a side stream, with a workspace that grows between."""
    budget = CacheBudget(1, 3, Hkv, 40 * BS)
    pool = Pool(3, 40, 90, Hkv, BS, D, 1)
    kc, vc = pool.caches[0]
    pool.fork([-1, -1, -1], [0, 1, 2], [0, 0, 0], [20, 500, 64])
    side = torch.cuda.Stream()
    passes = []
    for row, n in ((0, 20), (1, 500)):
        q = torch.randn((n, Hq, D), generator=torch.Generator("cuda").manual_seed(n), device="cuda").bfloat16()
        p = PromptPass(q, kc, vc, pool.table[row:row + 1], ints([0, n]), ints([0]), n, 0, 0.125)
        p.run(tuple(torch.randn((n, Hkv, D), device="cuda").bfloat16() for _ in range(2)))
        passes.append((row, p))
    move = ints([1]), ints([2]), ints([500])  # they live as long as the call
    side.wait_stream(torch.cuda.current_stream())
    for row, p in passes:
        budget.observe_prompt(0, p, row=row, stream=side)
    slots, new_len, st = budget.evict(pool.k, pool.v, pool.table, BS, 90, *move, 64, 4, 8, D, S.SPEC_BF16, stream=side)
    side.synchronize()
    assert st.tolist() == [0] and new_len.tolist() == [64]
    for row, p in passes:
        d = dict(q=p.q, k=kc, table=pool.table[row:row + 1], seq_off=p.seq_off, prefix=p.prefix_len, Hq=Hq, Hkv=Hkv, D=D, bs=BS, scale=0.125, stride=40 * BS)
        _weights_hold(budget, 0, row, None, d)
    for h in range(Hkv):
        assert slots[0, 0, h].tolist() == keep_reference(budget.weight[0, 1, h].tolist(), 500, 64, 4, 8)
