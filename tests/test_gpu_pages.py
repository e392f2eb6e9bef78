"""Pages of the cache: pa_copy_blocks, pa_tree_commit, and pa_fork_sequences / pa_grow_sequences /
pa_free_sequences against plain Python, with every refusal leaving all arrays as they were."""
import random

import pytest
import torch

from tests.spec_reference import Pages

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from paged_kv_cache_31_gb300 import binding

    assert binding.pa_device_status() == binding.PA_OK
    return binding


def _i32(x, *shape):
    t = torch.tensor(x, dtype=torch.int32, device=DEV)
    return t.view(*shape) if shape else t


def _pool(seed, NB, bs, Hkv, D, dtype):
    gen = torch.Generator().manual_seed(seed)
    return (torch.randn(NB, bs, Hkv, D, generator=gen) * 4).to(dtype).to(DEV)


def _bytes(t):
    return t.contiguous().view(torch.uint8)


# ---- copies -----------------------------------------------------------------------------------


@pytest.mark.parametrize("dtype", [BF16, F32, E4M3])
@pytest.mark.parametrize("n", [1, 2, 255, 256, 257, 700])
def test_copy_blocks(pa, n, dtype):
    NB = 2 * n + 5
    gen = torch.Generator().manual_seed(n)
    ids = torch.randperm(NB, generator=gen)
    dst, rest = ids[:n], ids[n:]
    src = rest[torch.randint(0, len(rest), (n,), generator=gen)]
    pairs = torch.stack([src, dst], 1).int()
    pairs[::7] = -1
    kb, vb = _pool(1, NB, 16, 2, 64, dtype), _pool(2, NB, 16, 2, 64, dtype)
    wk, wv = _bytes(kb).clone(), _bytes(vb).clone()
    live = pairs[:, 0] >= 0
    s, d = pairs[live, 0].long().to(DEV), pairs[live, 1].long().to(DEV)
    wk[d], wv[d] = wk[s], wv[s]
    pa.pa_copy_blocks(kb, vb, pairs.to(DEV))
    assert pa.pa_device_status() == pa.PA_OK
    assert torch.equal(_bytes(kb), wk) and torch.equal(_bytes(vb), wv)


@pytest.mark.parametrize("bs,Hkv,D", [(1, 3, 1), (5, 1, 7), (16, 8, 128), (3, 5, 6), (64, 8, 128)])
def test_copy_odd_blocks_and_one_pool(pa, bs, Hkv, D):
    for dtype in (BF16, E4M3, F32):
        kb = _pool(3, 9, bs, Hkv, D, dtype)
        want = _bytes(kb).clone()
        want[[4, 7]] = want[[0, 0]]
        pa.pa_copy_blocks(kb, None, _i32([[0, 4], [-1, -1], [0, 7]]))
        assert pa.pa_device_status() == pa.PA_OK
        assert torch.equal(_bytes(kb), want)


def test_copy_block_factors(pa):
    """Per-block dequantisation factors move with the same pairs."""
    ks, vs = torch.rand(10, 4, device=DEV), torch.rand(10, 4, device=DEV)
    wk, wv = ks.clone(), vs.clone()
    wk[3], wv[3] = ks[8], vs[8]
    pa.pa_copy_blocks(ks.view(10, 1, 4, 1), vs.view(10, 1, 4, 1), _i32([[8, 3]]))
    assert pa.pa_device_status() == pa.PA_OK
    assert torch.equal(ks, wk) and torch.equal(vs, wv)


@pytest.mark.parametrize("n", [8, 300])
def test_copy_refusals_write_nothing(pa, n):
    NB = 2 * n
    base = [[i, n + i] for i in range(n)]
    kb, vb = _pool(4, NB, 16, 1, 64, BF16), _pool(5, NB, 16, 1, 64, BF16)
    wk, wv = kb.clone(), vb.clone()
    for at, pair in ((3, [NB, n + 3]), (3, [0, NB]), (n - 1, [-1, 5]), (0, [4, -1]), (0, [-2, -2]),
                     (2, [2, n + 5]),          # the same destination twice
                     (2, [2, 1]),              # a destination that is a source
                     (5, [n + 5, n + 5])):     # onto itself
        pairs = [list(p) for p in base]
        pairs[at] = pair
        pa.pa_copy_blocks(kb, vb, _i32(pairs))
        assert pa.pa_device_status() == pa.PA_EINVAL, (at, pair)
        assert torch.equal(kb, wk) and torch.equal(vb, wv)
    pa.pa_copy_blocks(kb, vb, torch.empty(0, 2, dtype=torch.int32, device=DEV))
    assert pa.pa_device_status() == pa.PA_OK and torch.equal(kb, wk)


# ---- accepted rows ----------------------------------------------------------------------------


def _commit_case(S, n, most, ctx_hi, bs, seed):
    rng = random.Random(seed)
    ctx = [rng.randint(0, ctx_hi) for _ in range(S)]
    need = [-(-(c + n) // bs) for c in ctx]
    NB = sum(need) + 1
    ids = list(range(NB))
    rng.shuffle(ids)
    tables, at = [], 0
    for k in need:
        tables.append(ids[at:at + k] + [0] * (max(need) - k))
        at += k
    count = [rng.randint(0, most) for _ in range(S)]
    acc = [sorted(rng.sample(range(n), c)) + [rng.randint(-5, n) for _ in range(most - c)]
           for c in count]
    return ctx, NB, tables, count, acc


@pytest.mark.parametrize("dtype,Hkv,D", [(BF16, 8, 128), (E4M3, 2, 128), (F32, 1, 64), (BF16, 1, 7),
                                         (E4M3, 3, 5)])
@pytest.mark.parametrize("S,n,most,bs", [(1, 24, 4, 16), (5, 64, 30, 16), (1, 1, 1, 16),
                                         (300, 40, 9, 16), (4, 33, 33, 5)])
def test_commit(pa, S, n, most, bs, dtype, Hkv, D):
    ctx, NB, tables, count, acc = _commit_case(S, n, most, 70, bs, S + n)
    kb, vb = _pool(6, NB, bs, Hkv, D, dtype), _pool(7, NB, bs, Hkv, D, dtype)
    k0, v0 = kb.clone(), vb.clone()
    wk, wv = kb.clone(), vb.clone()
    row = lambda p: _bytes(p).view(NB * bs, -1)  # noqa: E731
    to, frm = [], []
    for s in range(S):
        slot = lambda p: tables[s][p // bs] * bs + p % bs  # noqa: E731,B023
        for i in range(count[s]):
            to.append(slot(ctx[s] + i))
            frm.append(slot(ctx[s] + acc[s][i]))
    if to:
        row(wk)[to], row(wv)[to] = row(k0)[frm], row(v0)[frm]
    pa.pa_tree_commit(kb, vb, _i32(tables), _i32(ctx), _i32(acc, S, most), _i32(count))
    assert pa.pa_device_status() == pa.PA_OK
    assert torch.equal(_bytes(kb), _bytes(wk)) and torch.equal(_bytes(vb), _bytes(wv))


@pytest.mark.parametrize("S", [3, 400])
def test_commit_refusals_write_nothing(pa, S):
    ctx, NB, tables, count, acc = _commit_case(S, 30, 6, 50, 16, 5)
    count[1] = 4
    acc[1] = [2, 5, 9, 20, 0, 0]
    kb, vb = _pool(8, NB, 16, 2, 64, BF16), _pool(9, NB, 16, 2, 64, BF16)
    wk, wv = kb.clone(), vb.clone()

    def run(tables=tables, ctx=ctx, acc=acc, count=count):
        pa.pa_tree_commit(kb, vb, _i32(tables), _i32(ctx), _i32(acc), _i32(count))
        assert pa.pa_device_status() == pa.PA_EINVAL
        assert torch.equal(kb, wk) and torch.equal(vb, wv)

    def put(rows, s, value):
        rows = [list(r) if isinstance(r, list) else r for r in rows]
        rows[s] = value
        return rows

    run(acc=put(acc, 1, [2, 5, 5, 20, 0, 0]))       # the same node twice
    run(acc=put(acc, 1, [5, 2, 9, 20, 0, 0]))       # not increasing
    run(acc=put(acc, 1, [-1, 2, 9, 20, 0, 0]))
    run(acc=put(acc, 1, [2, 5, 9, 10 ** 6, 0, 0]))  # beyond the table
    run(acc=put(acc, 1, [2, 5, 9, 2 ** 31 - 1, 0, 0]))
    run(count=put(count, 1, 7))
    run(count=put(count, 1, -1))
    run(ctx=put(ctx, 1, -1))
    run(ctx=put(ctx, 1, 2 ** 31 - 1))
    bad = (ctx[1] + 9) // 16
    run(tables=put(tables, 1, tables[1][:bad] + [NB] + tables[1][bad + 1:]))


# ---- bookkeeping ------------------------------------------------------------------------------


class State:
    """The device arrays of a Pages object, with `spare` unused entries in the free list."""

    def __init__(self, p):
        self.p = p
        self.tables, self.lens = _i32(p.tables), _i32(p.lens)
        self.refs = _i32(p.refs)
        self.free = _i32(p.free + [-3] * (len(p.refs) - len(p.free)))
        self.count = _i32([len(p.free)])

    def args(self):
        return self.refs, self.free, self.count, self.p.block

    def arrays(self):
        return self.tables, self.lens, self.refs, self.free, self.count

    def same(self):
        p = self.p
        assert self.tables.tolist() == p.tables
        assert self.lens.tolist() == p.lens
        assert self.refs.tolist() == p.refs
        assert self.count.item() == len(p.free)
        assert self.free[:len(p.free)].tolist() == p.free


def _state(rows, cols, lens, block, seed, extra):
    """`lens` sequences with blocks of their own, then empty rows; a shuffled free list."""
    rng = random.Random(seed)
    need = [-(-n // block) for n in lens]
    NB = sum(need) + extra
    ids = list(range(NB))
    rng.shuffle(ids)
    tables, refs, at = [], [0] * NB, 0
    for r in range(rows):
        k = need[r] if r < len(lens) else 0
        tables.append(ids[at:at + k] + [rng.randint(-9, 9) for _ in range(cols - k)])
        for b in ids[at:at + k]:
            refs[b] = 1
        at += k
    return State(Pages(tables, lens + [0] * (rows - len(lens)), refs, ids[at:], block))


@pytest.mark.parametrize("block", [16, 1, 5])
@pytest.mark.parametrize("lens,forks", [([40], 3), ([32, 17, 0, 1], 9), ([700, 15], 40),
                                        ([4000, 4097, 9], 300)])
def test_fork_grow_free(pa, lens, forks, block):
    if block == 1 and forks > 100:
        lens = [n // 8 for n in lens]
    rng = random.Random(forks + block)
    P, cols = len(lens), -(-max(lens) // block) + 8
    st = _state(P + forks, cols, lens, block, 3, forks * 9 + 4)
    kids = list(range(P, P + forks))
    rng.shuffle(kids)
    par = [rng.randrange(P) for _ in kids]
    pairs = pa.pa_fork_sequences(st.tables, st.lens, _i32(par), _i32(kids), *st.args())
    assert [tuple(x) for x in pairs.tolist()] == st.p.fork(par, kids)
    assert pa.pa_device_status() == pa.PA_OK
    st.same()
    rows = rng.sample(range(P + forks), P + forks)
    new = [min(cols * block, st.p.lens[r] + rng.randint(0, 5 * block)) for r in rows]
    pa.pa_grow_sequences(st.tables, st.lens, _i32(rows), _i32(new), *st.args())
    st.p.grow(rows, new)
    st.same()
    some = rng.sample(range(P + forks), (P + forks) // 2)
    pa.pa_free_sequences(st.tables, st.lens, _i32(some), *st.args())
    st.p.end(some)
    st.same()
    rest = [r for r in range(P + forks) if r not in some]
    pa.pa_free_sequences(st.tables, st.lens, _i32(rest), *st.args())
    st.p.end(rest)
    st.same()
    assert pa.pa_device_status() == pa.PA_OK
    assert not any(st.p.refs) and len(st.p.free) == len(st.p.refs)


@pytest.mark.parametrize("block", [16, 1, 5])
def test_trim(pa, block):
    """Rows cut to nothing, inside a block, at a block's end, not at all; shared and own blocks."""
    rng = random.Random(block)
    lens = [40, 16, 0, 1, 333, 80, 7]
    st = _state(9, 70 if block > 1 else 340, lens, block, 9, 120)
    pairs = pa.pa_fork_sequences(st.tables, st.lens, _i32([4, 0]), _i32([7, 8]), *st.args())
    assert [tuple(x) for x in pairs.tolist()] == st.p.fork([4, 0], [7, 8])
    rows = [4, 0, 1, 2, 3, 7, 8, 5]
    for new in ([330, 40, 16, 0, 0, 321, 1, 75], [0, 39, 0, 0, 0, 320, 0, 16]):
        order = rng.sample(range(len(rows)), len(rows))
        r, n = [rows[i] for i in order], [min(new[i], st.p.lens[rows[i]]) for i in order]
        pa.pa_trim_sequences(st.tables, st.lens, _i32(r), _i32(n), *st.args())
        st.p.end(r, n)
        st.same()
    old = [st.p.lens[r] for r in (0, 5)]
    for r, n in (([0], [old[0] + 1]), ([0], [-1]), ([0, 0], [0, 0]), ([9], [0]), ([5, 0], [0, 100])):
        _refused(pa, st, lambda: pa.pa_trim_sequences(st.tables, st.lens, _i32(r), _i32(n),  # noqa: B023
                                                      *st.args()))
    pa.pa_free_sequences(st.tables, st.lens, _i32(list(range(9))), *st.args())
    st.p.end(range(9))
    st.same()
    assert pa.pa_device_status() == pa.PA_OK and not any(st.p.refs)


def test_more_rows_than_one_round(pa):
    """Lists longer than the 1024 rows that the kernel takes at a time."""
    lens = [33, 16, 5]
    n = 2500
    st = _state(3 + n, 4, lens, 16, 4, 3 * n)
    par = [i % 3 for i in range(n)]
    kids = list(range(3, 3 + n))
    pairs = pa.pa_fork_sequences(st.tables, st.lens, _i32(par), _i32(kids), *st.args())
    assert [tuple(x) for x in pairs.tolist()] == st.p.fork(par, kids)
    st.same()
    new = [min(64, st.p.lens[k] + k % 20) for k in kids]
    pa.pa_grow_sequences(st.tables, st.lens, _i32(kids), _i32(new), *st.args())
    st.p.grow(kids, new)
    st.same()
    new = [n // 3 for n in new]
    pa.pa_trim_sequences(st.tables, st.lens, _i32(kids), _i32(new), *st.args())
    st.p.end(kids, new)
    st.same()
    pa.pa_free_sequences(st.tables, st.lens, _i32(kids[::-1]), *st.args())
    st.p.end(kids)
    st.same()
    assert pa.pa_device_status() == pa.PA_OK


def test_large_pool(pa):
    """Freed ids from all over a large pool come back in ascending order."""
    NB = 300_001
    gen = torch.Generator().manual_seed(5)
    ids = torch.randperm(NB, generator=gen)
    tables = ids[:64 * 1000].view(64, 1000).int().to(DEV)
    lens = torch.full((64,), 16000, dtype=torch.int32, device=DEV)
    refs = torch.zeros(NB, dtype=torch.int32, device=DEV)
    refs[ids[:64000].to(DEV)] = 1
    refs[tables[0].long()] += 1  # held by someone else too
    free = torch.full((NB,), -1, dtype=torch.int32, device=DEV)
    count = torch.zeros(1, dtype=torch.int32, device=DEV)
    rows = torch.arange(64, dtype=torch.int32, device=DEV)
    pa.pa_free_sequences(tables, lens, rows, refs, free, count, 16)
    assert pa.pa_device_status() == pa.PA_OK
    assert count.item() == 63000 and not lens.any()
    assert torch.equal(free[:63000].cpu().long(), ids[1000:64000].sort().values)
    assert (free[63000:] == -1).all()
    assert refs.sum().item() == 1000


def _refused(pa, st, f):
    before = [x.clone() for x in st.arrays()]
    f()
    assert pa.pa_device_status() == pa.PA_EINVAL
    for x, y in zip(st.arrays(), before):
        assert torch.equal(x, y)


def test_bookkeeping_refusals_leave_everything(pa):
    st = _state(8, 6, [40, 16, 3], 16, 6, 4)
    NB = len(st.p.refs)
    pairs = torch.full((2, 2), 77, dtype=torch.int32, device=DEV)

    def fork(par, kids):
        pa.pa_fork_sequences(st.tables, st.lens, _i32(par), _i32(kids), *st.args(),
                             block_pairs=pairs[:len(par)])
        assert (pairs == 77).all()

    def grow(rows, new):
        pa.pa_grow_sequences(st.tables, st.lens, _i32(rows), _i32(new), *st.args())

    def free(rows):
        pa.pa_free_sequences(st.tables, st.lens, _i32(rows), *st.args())

    _refused(pa, st, lambda: fork([0, 1], [4, 4]))       # one child twice
    _refused(pa, st, lambda: fork([0, 4], [4, 5]))       # a child that is a parent
    _refused(pa, st, lambda: fork([0], [0]))
    _refused(pa, st, lambda: fork([8], [4]))
    _refused(pa, st, lambda: fork([0], [-1]))
    _refused(pa, st, lambda: grow([0], [39]))            # shorter
    _refused(pa, st, lambda: grow([0, 0], [41, 42]))
    _refused(pa, st, lambda: grow([0], [97]))            # beyond the table
    _refused(pa, st, lambda: grow([3, 4], [48, 32]))     # five blocks of four
    _refused(pa, st, lambda: free([1, 1]))
    _refused(pa, st, lambda: free([-1]))
    _refused(pa, st, lambda: free([8]))

    def broken(array, at, value, f):
        old = array[at].clone()
        array[at] = value
        _refused(pa, st, f)
        array[at] = old

    broken(st.tables, (0, 1), NB, lambda: fork([0], [4]))
    broken(st.tables, (0, 1), -1, lambda: free([0]))
    broken(st.lens, 0, -1, lambda: free([0]))
    broken(st.lens, 0, 97, lambda: fork([0], [4]))
    broken(st.refs, st.p.tables[0][0], 0, lambda: fork([0], [4]))
    broken(st.refs, st.p.tables[0][0], 0, lambda: free([2, 0, 1]))  # a double free is undone
    broken(st.refs, st.p.free[-1], 1, lambda: fork([0], [4]))       # not free
    broken(st.free, len(st.p.free) - 1, NB, lambda: grow([3], [1]))
    broken(st.free, len(st.p.free) - 1, -1, lambda: fork([0], [4]))
    broken(st.count, 0, -1, lambda: free([0]))
    broken(st.count, 0, NB + 1, lambda: grow([0], [41]))
    broken(st.count, 0, NB, lambda: free([1]))                      # the list would overflow
    broken(st.count, 0, 0, lambda: fork([0], [4]))                  # nothing to take
    # and all of it still works
    got = pa.pa_fork_sequences(st.tables, st.lens, _i32([0, 1]), _i32([4, 5]), *st.args())
    assert [tuple(x) for x in got.tolist()] == st.p.fork([0, 1], [4, 5])
    st.same()
    pa.pa_free_sequences(st.tables, st.lens, _i32([0, 4, 5, 1, 2]), *st.args())
    st.p.end([0, 4, 5, 1, 2])
    st.same()
    assert pa.pa_device_status() == pa.PA_OK


def test_an_earlier_error_stops_every_call(pa):
    st = _state(4, 4, [20], 16, 7, 4)
    kb = _pool(1, len(st.p.refs), 16, 1, 64, BF16)
    want = kb.clone()
    before = [x.clone() for x in st.arrays()]
    pa.pa_copy_blocks(kb, None, _i32([[0, 99]]))  # recorded
    pa.pa_fork_sequences(st.tables, st.lens, _i32([0]), _i32([1]), *st.args())
    pa.pa_grow_sequences(st.tables, st.lens, _i32([0]), _i32([40]), *st.args())
    pa.pa_free_sequences(st.tables, st.lens, _i32([0]), *st.args())
    pa.pa_copy_blocks(kb, None, _i32([[0, 1]]))
    pa.pa_tree_commit(kb, kb.clone(), _i32([[0, 1]]), _i32([0]), _i32([[3]]), _i32([1]))
    assert pa.pa_device_status() == pa.PA_EINVAL
    assert torch.equal(kb, want)
    for x, y in zip(st.arrays(), before):
        assert torch.equal(x, y)


def test_bookkeeping_in_a_graph_in_front_of_attention(pa):
    """Fork, copy and attend captured together: the attention's planner, which may start early,
    sees the tables that the fork in front of it writes."""
    st = _state(3, 8, [75, 40], 16, 8, 20)
    NB = len(st.p.refs)
    kb, vb = _pool(11, NB, 16, 2, 128, BF16), _pool(12, NB, 16, 2, 128, BF16)
    q = torch.randn(1, 8, 128, device=DEV).to(BF16)
    out, want = torch.empty_like(q), torch.empty_like(q)
    par, kid = _i32([0]), _i32([2])
    pairs = torch.empty(1, 2, dtype=torch.int32, device=DEV)
    qsl, pos = _i32([0, 1]), _i32([0])
    ws = pa.workspace_for(q, kb, qsl, st.tables[2:])

    def step():
        pa.pa_fork_sequences(st.tables, st.lens, par, kid, *st.args(), block_pairs=pairs)
        pa.pa_copy_blocks(kb, vb, pairs)
        pa.pa_varlen_forward(q, kb, vb, out, qsl, st.lens[2:], pos, st.tables[2:], 0.1,
                             causal=False, workspace=ws)
        pa.pa_free_sequences(st.tables, st.lens, kid, *st.args())

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for p in (1, 0, 1):
        par.fill_(p)
        out.zero_()
        g.replay()
        pa.pa_varlen_forward(q, kb, vb, want, qsl, st.lens[p:p + 1], pos,
                             st.tables[p:p + 1].contiguous(), 0.1, causal=False)
        assert torch.equal(out, want)
    assert pa.pa_device_status() == pa.PA_OK
