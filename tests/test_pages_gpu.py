"""The page calls through the C ABI against plain Python on lists: tables,
pools, counts, statuses and every byte of every layer's caches."""
import numpy as np
import pytest
import torch

import tree_speculative_verification_spec_gb300 as S
from request_life import Pages

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from tree_speculative_verification_spec_gb300 import build
    build.build()
    S.lib()


class Both:
    """The same state on the device and as the plain reference."""

    def __init__(self, table, pool, count, num_blocks, bs, layers=0, Hkv=2, D=64, dtype=torch.bfloat16, seed=0):
        self.B, self.mb, self.nb, self.bs, self.layers, self.Hkv, self.D = len(table), len(table[0]), num_blocks, bs, layers, Hkv, D
        kind = np.int16 if dtype == torch.bfloat16 else np.int32
        g = np.random.default_rng(seed)
        caches = [g.integers(0, 30000, (num_blocks, Hkv, bs, D)).astype(kind) for _ in range(2 * layers)]
        self.code = S.SPEC_BF16 if dtype == torch.bfloat16 else S.SPEC_F32
        self.dev = [torch.from_numpy(c.copy()).cuda() for c in caches]
        ptr = lambda part: torch.tensor([t.data_ptr() for t in part], dtype=torch.int64, device="cuda") if layers else None  # noqa: E731
        self.k, self.v = ptr(self.dev[0::2]), ptr(self.dev[1::2])
        self.ref = Pages(table, pool, count, num_blocks, bs, caches)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.table, self.pool, self.count = torch.tensor(table, **i32), torch.tensor(pool, **i32), torch.tensor([count], **i32)

    def ws(self, n):
        return torch.full((S.spec_pages_workspace_size(self.B, self.mb, self.nb, n),), 255, dtype=torch.uint8, device="cuda")

    def ints(self, v):
        return torch.tensor(v, dtype=torch.int32, device="cuda")

    def fork(self, src, dst, length, room):
        n = len(src)
        st = torch.full((n,), 77, dtype=torch.int32, device="cuda")
        S.spec_pages_fork(self.k, self.v, self.layers, self.table, self.B, self.mb, self.bs, self.nb, self.ints(src), self.ints(dst),
                          self.ints(length), self.ints(room), n, self.Hkv, self.D, self.code, self.pool, self.count, self.ws(n), st)
        want = self.ref.fork(list(src), list(dst), list(length), list(room))
        assert st.tolist() == want
        self.same()
        return want

    def free(self, rows, keep=None):
        n = len(rows)
        st = torch.full((n,), 77, dtype=torch.int32, device="cuda")
        S.spec_pages_free(self.table, self.B, self.mb, self.bs, self.nb, self.ints(rows), None if keep is None else self.ints(keep), n,
                          self.pool, self.count, self.ws(n), st)
        want = self.ref.free(list(rows), [0] * n if keep is None else list(keep))
        assert st.tolist() == want
        self.same()
        return want

    def compact(self):
        st, moved = self.ints([77]), self.ints([77])
        page_map = torch.full((self.nb,), 77, dtype=torch.int32, device="cuda")
        S.spec_pages_compact(self.k, self.v, self.layers, self.table, self.B, self.mb, self.bs, self.nb, self.Hkv, self.D, self.code,
                             self.pool, self.count, page_map, moved, self.ws(0), st)
        want, to, n = self.ref.compact()
        assert st.item() == want and moved.item() == n and page_map.tolist() == to
        self.same()
        return want, n

    def same(self):
        assert self.count.item() == self.ref.count
        assert self.pool.tolist() == self.ref.pool
        assert self.table.tolist() == self.ref.table
        for got, want in zip(self.dev, self.ref.caches):
            assert np.array_equal(got.cpu().numpy(), want)


def _empty(B, mb):
    return [[-1] * mb for _ in range(B)]


@pytest.mark.parametrize("dtype,D,bs,Hkv,layers", [(torch.bfloat16, 64, 8, 2, 3), (torch.float32, 128, 16, 1, 1),
                                                   (torch.bfloat16, 128, 64, 3, 2), (torch.bfloat16, 64, 256, 1, 1),
                                                   (torch.bfloat16, 64, 16, 2, 0)])
def test_a_life_of_forks_frees_and_compactions(dtype, D, bs, Hkv, layers):
    g = np.random.default_rng(D + bs)
    B, mb, nb = 12, 9, 70
    order = g.permutation(nb).tolist()
    caller = order[:4]  # ids in neither table nor pool: the caller's own
    s = Both(_empty(B, mb), order[4:] + [-1] * 6, nb - 4, nb, bs, layers, Hkv, D, dtype)
    assert s.fork([-1, -1, -1], [0, 1, 2], [0, 0, 0], [3 * bs + 1, 1, 0]) == [0, 0, 0]
    lens = {0: 3 * bs + 1, 1: 1}
    assert s.fork([0, 0, 1, 0], [3, 4, 5, 6], [3 * bs + 1, 2 * bs, 1, 5], [0, bs, 2 * bs, 0]) == [0] * 4
    assert s.fork([0, 3], [0, 7], [3 * bs + 1, 2 * bs + bs // 2], [4 * bs, 3]) == [0, 0]  # a row extended, another forked
    s.free([4, 6], [bs, 0])
    s.compact()
    s.fork([7, 5], [8, 9], [2 * bs + 1, 1], [1, 0])
    s.free([0, 3, 7, 8])
    _, moved = s.compact()
    s.free(list(range(B)))
    assert s.count.item() == nb - 4 and sorted(s.pool.tolist()[:nb - 4] + caller) == list(range(nb))
    assert s.compact() == (0, 0)


@pytest.mark.parametrize("seed", range(6))
def test_random_lives(seed):
    g = np.random.default_rng(100 + seed)
    B, mb, bs = int(g.integers(2, 40)), int(g.integers(1, 40)), int(g.choice([8, 16]))
    nb = int(g.integers(5, B * mb + 20))
    s = Both(_empty(B, mb), g.permutation(nb).tolist(), nb, nb, bs, 1, 1, 64, torch.bfloat16, seed)
    held = {}
    for _ in range(12):
        op = g.integers(0, 4)
        free_rows = [r for r in range(B) if r not in held]
        if op <= 1 and free_rows:
            n = int(g.integers(1, len(free_rows) + 1))
            dst = g.choice(free_rows, n, replace=False).tolist()
            src, length, room = [], [], []
            for _ in dst:
                r = int(g.choice(list(held))) if held and g.random() < 0.8 else -1
                top = held.get(r, 0)
                src.append(r)
                length.append(int(g.integers(0, top + 1)))
                room.append(int(g.integers(0, 3 * bs)))
            st = s.fork(src, dst, length, room)
            for r, k, m, t in zip(dst, length, room, st):
                if t == 0:
                    held[r] = k + m
        elif op == 2 and held:
            rows = g.choice(list(held), int(g.integers(1, len(held) + 1)), replace=False).tolist()
            keep = [int(g.integers(0, held[r] + 1)) for r in rows]
            for r, k, t in zip(rows, keep, s.free(rows, keep)):
                if t == 0:
                    held[r] = k
                    if k == 0:
                        del held[r]
        else:
            assert s.compact()[0] == 0


def test_fork_refusals():
    bs, mb, nb = 8, 4, 40
    table = [[0, 1, 2, -1], [3, -1, -1, -1], [-1] * 4, [-1] * 4, [40, 5, -1, -1], [-1] * 4, [-1] * 4, [6, 7, 8, 9]]
    pool = list(range(10, 20)) + [-1] * 5
    s = Both(table, pool, 10, nb, bs, 1)
    # one call with every kind of bad row
    assert s.fork([0, 8, 0, 0, 0, -1, 7], [2, 3, -1, 8, 5, 6, 7], [9, 1, 1, 1, -1, 2, 32], [0] * 7) == [0, 128, 128, 128, 128, 128, 0]
    s = Both(table, pool, 10, nb, bs, 1)
    assert s.fork([0], [1], [8], [0]) == [S.SPEC_DEV_BAD_ROW]               # the row holds a page where one would go
    assert s.fork([4], [2], [9], [0]) == [S.SPEC_DEV_BAD_BLOCK]             # a source page out of range
    assert s.fork([0], [2], [25], [8]) == [S.SPEC_DEV_CAPACITY]             # more slots than a row has
    assert s.fork([2], [3], [1], [0]) == [S.SPEC_DEV_BAD_BLOCK]             # the source has no such page
    assert s.fork([0, 0], [2, 2], [8, 8], [0, 0]) == [S.SPEC_DEV_BAD_ROW] * 2
    assert s.fork([0, 2], [2, 3], [8, 8], [0, 0]) == [0, S.SPEC_DEV_BAD_ROW]  # a chain within one call
    # a short pool: the forks that need no page still go through
    s = Both(table, pool, 2, nb, bs, 1)
    assert s.fork([0, 0, 0], [2, 3, 5], [9, 16, 17], [0, 0, 8]) == [S.SPEC_DEV_CAPACITY, 0, S.SPEC_DEV_CAPACITY]
    s = Both(table, [10, 99, 11], 3, nb, bs, 1)                             # a pool entry that is no page
    assert s.fork([0], [2], [9], [0]) == [0]
    assert s.fork([0], [3], [9], [0]) == [S.SPEC_DEV_BAD_BLOCK]
    for count in (-1, 4):
        s = Both(table, [10, 11, 12], count, nb, bs, 1)
        assert s.fork([0, 0], [2, 3], [9, 8], [0, 0]) == [S.SPEC_DEV_CAPACITY, 0]


def test_free_refusals():
    table = [[0, 1, 2, -1], [0, 3, -1, -1], [40, 4, -1, -1], [5, 6, 7, 8]]
    s = Both(table, [20, -1, -1, -1, -1, -1, -1, -1], 1, 40, 8)
    assert s.free([0, 4, -1, 3, 3, 2]) == [0, 128, 128, 128, 128, 16]
    assert s.free([1], [-1]) == [128]
    assert s.free([3], [9]) == [0]
    assert s.free([2], [8]) == [0]          # the bad entry is kept, not dropped
    s = Both(table, [20, 21, -1], 2, 40, 8)
    assert s.free([0, 1]) == [4, 4]         # pages 1, 2, 0 and 3: the pool has room for one
    assert s.free([1], [8]) == [0]
    s = Both(table, [20, 21], 2, 40, 8)
    assert s.free([1], [16]) == [0]         # nothing to release


def test_compact_refusals():
    for table, pool, count in (([[0, 40]], [1, 2], 2), ([[0, 1]], [2, 2], 2), ([[0, 1]], [1, 2], 2), ([[0, 1]], [2, -1], 2),
                               ([[0, 1]], [2, 40], 2), ([[0, 1]], [2, 3], 3), ([[0, 1]], [2, 3], -1)):
        s = Both(table, pool, count, 40, 8, 1)
        assert s.compact() == (16, 0)


def test_wide_tables():
    """Tables whose passes take several rounds of the plan's cluster."""
    g = np.random.default_rng(7)
    B, mb, bs = 300, 128, 8
    nb = B * mb
    ids = g.permutation(nb).reshape(B, mb)
    table = np.where(g.random((B, mb)) < 0.6, ids, -1)
    shared = g.integers(0, 30, B)
    table[30:, :40] = table[shared[30:], :40]
    held = set(table[table >= 0].tolist())
    pool = [p for p in g.permutation(nb).tolist() if p not in held]
    s = Both(table.tolist(), pool + [-1] * (nb - len(pool)), len(pool), nb, bs)
    s.free(g.choice(B, 170, replace=False).tolist())
    s.free([int(r) for r in range(0, 300, 3)], [int(k) for k in g.integers(0, mb * bs, 100)])
    s.compact()


def test_page_calls_replay_from_a_graph():
    bs, nb = 16, 50
    s = Both([[0, 1, 2, -1]] + _empty(3, 4), list(range(3, 40)), 37, nb, bs, 2)
    start = [t.clone() for t in (s.table, s.pool, s.count)]
    src, dst, length, room = s.ints([0, 0]), s.ints([1, 2]), s.ints([40, 33]), s.ints([5, 16])
    ws, st = s.ws(4), s.ints([0, 0])
    rows, keep = s.ints([1]), s.ints([16])
    st1, st2, moved, page_map = s.ints([0]), s.ints([0]), s.ints([0]), torch.zeros(nb, dtype=torch.int32, device="cuda")

    def life():
        S.spec_pages_fork(s.k, s.v, 2, s.table, 4, 4, bs, nb, src, dst, length, room, 2, s.Hkv, s.D, s.code, s.pool, s.count, ws, st)
        S.spec_pages_free(s.table, 4, 4, bs, nb, rows, keep, 1, s.pool, s.count, ws, st1)
        S.spec_pages_compact(s.k, s.v, 2, s.table, 4, 4, bs, nb, s.Hkv, s.D, s.code, s.pool, s.count, page_map, moved, ws, st2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        life()
    assert torch.equal(s.table, start[0])
    graph.replay()
    assert s.ref.fork([0, 0], [1, 2], [40, 33], [5, 16]) == [0, 0]
    assert s.ref.free([1], [16]) == [0]
    s.ref.compact()
    torch.cuda.synchronize()
    s.same()


@pytest.mark.parametrize("B", [8192, 8193, 20000])
def test_tables_of_many_rows(B):
    """Rows named twice, rows at both ends of a long table, and more entries than
    a cluster has threads."""
    bs, nb = 8, 12000
    s = Both(_empty(B, 2), list(range(nb)), nb, nb, bs, 0, 1, 64, torch.bfloat16)
    n = 9000
    dst = [(7 * i + 3) % B for i in range(n)]
    dst[5], dst[6], dst[7] = B - 1, B, -1
    dst[8] = dst[4000]
    s.fork([-1] * n, dst, [0] * n, [1 + i % 9 for i in range(n)])
    first = dst[1]
    s.fork([first, first, dst[8]], [0, 0, 1], [1, 1, 0], [0, 0, 0])
    s.free([B - 1, first, 0, 0, B] + [d for d in dst[20:3000]], [0, 1, 0, 0, 0] + [0] * 2980)


class AllOrNothing(Pages):
    """A free that the pool cannot take flags every row that had a page to drop,
    not only those whose pages would have been released."""

    def free(self, rows, keep):
        status = super().free(rows, keep)
        if any(s & S.SPEC_DEV_CAPACITY for s in status):
            for i, r in enumerate(rows):
                if status[i] == 0 and any(p >= 0 for p in self.table[r][-(-keep[i] // self.bs):]):
                    status[i] = S.SPEC_DEV_CAPACITY
        return status


def _tight(table, pool, count, nb, bs=8):
    s = Both(table, pool, count, nb, bs)
    s.ref = AllOrNothing(table, pool, count, nb, bs)
    return s


def test_a_full_pool_flags_every_row_that_keeps_pages_it_should_drop():
    s = _tight([[0, 1], [0, -1], [-1, -1]], [5, 6], 2, 40)
    assert s.free([0, 1, 2]) == [4, 4, 0]      # row 1's page would go with row 0's; row 2 has none
    s = _tight([[0, 1, 2], [0, 1, -1], [3, 0, -1], [3, -1, -1]], [5, 6, -1], 2, 40)
    assert s.free([0, 1, 2], [0, 8, 8]) == [4, 4, 4]
    assert s.free([1, 2], [8, 8]) == [0, 0]    # both dropped pages stay with row 0: nothing to release
    assert s.free([0]) == [4]                  # pages 1 and 2: the pool has room for one


@pytest.mark.parametrize("seed", range(4))
def test_random_frees_into_a_tight_pool(seed):
    g = np.random.default_rng(300 + seed)
    B, mb, bs = int(g.integers(20, 400)), int(g.integers(3, 60)), 8
    nb = B * mb
    ids = g.permutation(nb).reshape(B, mb)
    table = np.where(g.random((B, mb)) < 0.7, ids, -1)
    half = B // 2
    table[half:, :mb // 2] = table[g.integers(0, half, B - half)][:, :mb // 2]
    held = set(table[table >= 0].tolist())
    spare = [p for p in g.permutation(nb).tolist() if p not in held]
    s = _tight(table.tolist(), spare + [-1] * (len(held) // 3), len(spare), nb, bs)
    flagged = 0
    for _ in range(12):
        rows = g.choice(B, int(g.integers(1, B // 2 + 1)), replace=False).tolist()
        flagged += any(s.free(rows, [int(k) for k in g.integers(0, mb * bs, len(rows))]))
    assert flagged


def test_pages_beyond_32_bit_offsets():
    """Partial pages copied and whole ones moved at the end of caches of more than
    2^32 bytes."""
    Hkv, D, bs, layers = 2, 128, 64, 1
    nb = (1 << 32) // (Hkv * bs * D * 2) + 5
    caches = [torch.zeros((nb, Hkv, bs, D), dtype=torch.int16, device="cuda") for _ in range(2)]
    rows = [torch.randint(0, 30000, (2, Hkv, bs, D), dtype=torch.int16, device="cuda") for _ in range(2)]
    for c, r in zip(caches, rows):
        c[nb - 4], c[nb - 3] = r[0], r[1]
    k, v = (torch.tensor([c.data_ptr()], dtype=torch.int64, device="cuda") for c in caches)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, pool, count = i([[nb - 4, nb - 3], [-1, -1]]), i([3, nb - 1]), i([2])
    ws = torch.empty(S.spec_pages_workspace_size(2, 2, nb, 1), dtype=torch.uint8, device="cuda")
    st, moved, page_map = i([77]), i([77]), torch.empty(nb, dtype=torch.int32, device="cuda")
    S.spec_pages_fork(k, v, layers, table, 2, 2, bs, nb, i([0]), i([1]), i([bs + 9]), None, 1, Hkv, D, S.SPEC_BF16, pool, count, ws, st)
    assert st.tolist() == [0] and table.tolist() == [[nb - 4, nb - 3], [nb - 4, nb - 1]] and count.tolist() == [1]
    for c, r in zip(caches, rows):
        assert torch.equal(c[nb - 1, :, :9], r[1, :, :9]) and not c[nb - 1, :, 9:].any()
    S.spec_pages_compact(k, v, layers, table, 2, 2, bs, nb, Hkv, D, S.SPEC_BF16, pool, count, page_map, moved, ws, st)
    assert st.tolist() == [0] and moved.tolist() == [1] and table.tolist() == [[nb - 4, nb - 3], [nb - 4, 3]] and pool.tolist()[0] == nb - 1
    for c, r in zip(caches, rows):
        assert torch.equal(c[3, :, :9], r[1, :, :9]) and torch.equal(c[nb - 4], r[0])


def test_calls_on_two_streams_at_once_with_their_own_tables():
    g = np.random.default_rng(17)
    ss = [Both(_empty(6, 9), g.permutation(60).tolist(), 60, 60, 8, 2, 2, 64, torch.bfloat16, i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in ss]
    st = [s.ints([77] * 3) for s in ss]
    ws = [s.ws(3) for s in ss]
    a = [[s.ints(x) for x in ([-1, -1, -1], [0, 1, 2], [0, 0, 0], [20, 33, 5])] for s in ss]
    b = [[s.ints(x) for x in ([0, 1, 1], [3, 4, 5], [17, 33, 8], [9, 0, 30])] for s in ss]
    gone = [s.ints([0, 4, 5]) for s in ss]
    torch.cuda.synchronize()
    for call in (a, b):
        for s, q, w, t, args in zip(ss, streams, ws, st, call):
            S.spec_pages_fork(s.k, s.v, s.layers, s.table, s.B, s.mb, s.bs, s.nb, *args, 3, s.Hkv, s.D, s.code, s.pool, s.count, w, t, stream=q)
    for s, q, w, t, rows in zip(ss, streams, ws, st, gone):
        S.spec_pages_free(s.table, s.B, s.mb, s.bs, s.nb, rows, None, 3, s.pool, s.count, w, t, stream=q)
    torch.cuda.synchronize()
    for s in ss:
        assert s.ref.fork([-1, -1, -1], [0, 1, 2], [0, 0, 0], [20, 33, 5]) == [0] * 3
        assert s.ref.fork([0, 1, 1], [3, 4, 5], [17, 33, 8], [9, 0, 30]) == [0] * 3
        assert s.ref.free([0, 4, 5], [0, 0, 0]) == [0] * 3
        s.same()
