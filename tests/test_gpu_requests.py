"""kv_resize_requests on the GPU against the plain implementation, entry for entry."""
import numpy as np
import pytest
import torch

import fp4_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkv():
    import paged_kv_cache_315_gb300 as m

    m.build()
    torch.cuda.set_device(0)
    m.pkv_device_error()
    return m


class Pool:
    """One set of arrays on both sides."""

    def __init__(self, B, MB, ring, head, count, bs, num_blocks, seed=0):
        rng = np.random.default_rng(seed)
        ids = rng.permutation(num_blocks).astype(np.int32)
        self.ring = np.full(ring, -5, np.int32)
        for i in range(min(count, num_blocks)):
            self.ring[(head + i) % ring] = ids[i]
        self.pool = np.array([head, count, 11, 12], np.int32)
        self.tables = np.full((B, MB), -7, np.int32)
        self.lens = np.zeros(B, np.int32)
        self.bs, self.num_blocks = bs, num_blocks
        self.dev = {k: torch.from_numpy(getattr(self, k).copy()).cuda()
                    for k in ("ring", "pool", "tables", "lens")}

    def step(self, pkv, target, rows, stream=None):
        target = np.asarray(target, np.int32)
        B = len(target)
        slots = torch.full((rows + 1,), -99, dtype=torch.int64, device="cuda")
        start = torch.full((B + 1,), -99, dtype=torch.int32, device="cuda")
        pkv.kv_resize_requests(self.dev["tables"], self.dev["lens"], torch.from_numpy(target).cuda(),
                               self.dev["ring"], self.dev["pool"], slots[:rows], start, self.bs,
                               self.num_blocks, stream=stream)
        got_err = pkv.pkv_device_error()
        want_slots, want_start, err = ref.resize(self.tables, self.lens, target, self.ring,
                                                 self.pool, rows, self.bs, self.num_blocks)
        assert got_err == err
        assert np.array_equal(slots[:rows].cpu().numpy(), want_slots)
        assert int(slots[rows]) == -99
        assert np.array_equal(start.cpu().numpy(), want_start)
        for k in ("ring", "pool", "tables", "lens"):
            assert np.array_equal(self.dev[k].cpu().numpy(), getattr(self, k)), k
        return want_slots, err


@pytest.mark.parametrize("B,MB,bs,seed", [(1, 4, 16, 1), (3, 7, 1, 2), (33, 9, 16, 3),
                                          (128, 40, 32, 4), (1500, 5, 64, 5), (5000, 3, 16, 6),
                                          (9000, 2, 16, 7)])
def test_random_steps(pkv, B, MB, bs, seed):
    rng = np.random.default_rng(seed)
    nb = B * MB
    p = Pool(B, MB, nb, int(rng.integers(nb)), nb, bs, nb, seed)
    cap = MB * bs
    for step in range(6):
        target = p.lens + rng.integers(0, max(2, cap // 3), B)
        target = np.where(rng.random(B) < 0.3, rng.integers(0, cap + 1, B), target)  # shrink or jump
        target = np.where(rng.random(B) < 0.1, 0, np.minimum(target, cap))
        rows = int(np.maximum(target - p.lens, 0).sum()) + int(rng.integers(0, 5))
        slots, err = p.step(pkv, target, rows)
        assert err == 0
        live = slots[slots >= 0]
        assert len(np.unique(live)) == len(live)
    # every block is free or in one table
    used = [int(x) for s in range(B) for x in p.tables[s, : -(-int(p.lens[s]) // bs)]]
    free = [int(p.ring[(p.pool[0] + i) % nb]) for i in range(p.pool[1])]
    assert sorted(used + free) == list(range(nb))


def test_decode_steps_one_token_each(pkv):
    B, bs = 130, 16
    p = Pool(B, 4, 4 * B, 0, 4 * B, bs, 4 * B)
    p.step(pkv, np.arange(B) % 50, int((np.arange(B) % 50).sum()))
    for _ in range(3):
        p.step(pkv, p.lens + 1, B)


def test_refused_growths(pkv):
    # 5 free blocks of 16: the third request's blocks do not fit; later ones that take blocks
    # are refused too, those that take none are not
    p = Pool(6, 8, 16, 14, 5, 16, 16)
    slots, err = p.step(pkv, [20, 10, 64, 1, 0, 3], 120)
    assert err == 32 and p.lens.tolist() == [20, 10, 0, 0, 0, 0]
    slots, err = p.step(pkv, [22, 12, 16, 0, 0, 16], 40)
    assert err == 0
    # too few rows: the first growth that does not fit and all behind it
    slots, err = p.step(pkv, [23, 14, 16, 0, 0, 16], 2)
    assert err == 32 and p.lens.tolist() == [23, 12, 16, 0, 0, 16]
    slots, err = p.step(pkv, [24, 12, 16, 0, 0, 16], 0)
    assert err == 32
    # nothing to do, and everything given back
    assert p.step(pkv, p.lens.copy(), 3)[1] == 0
    assert p.step(pkv, [0] * 6, 0)[1] == 0
    assert p.pool[1] == 5


def test_lengths_out_of_range(pkv):
    p = Pool(4, 2, 8, 0, 8, 16, 8)
    slots, err = p.step(pkv, [32, 33, -1, 5], 100)
    assert err == 8 and p.lens.tolist() == [32, 0, 0, 5]
    p.lens[0] = 1000
    p.dev["lens"][0] = 1000
    assert p.step(pkv, [3, 1, 1, 6], 10)[1] == 8


def test_pool_state_not_valid(pkv):
    for head, count in ((8, 1), (-1, 2), (0, 9), (3, -1)):
        p = Pool(2, 2, 8, 0, 8, 16, 8)
        p.pool[:2] = head, count
        p.dev["pool"][:2] = torch.tensor([head, count], dtype=torch.int32)
        assert p.step(pkv, [1, 0], 4)[1] == 32
        assert p.lens.tolist() == [0, 0]


def test_ring_shorter_than_what_returns(pkv):
    p = Pool(1, 6, 4, 2, 3, 1, 16)
    p.lens[0] = 5
    p.tables[0, :5] = [9, 8, 7, 6, 5]
    p.dev["lens"][0] = 5
    p.dev["tables"].copy_(torch.from_numpy(p.tables))
    assert p.step(pkv, [0], 0)[1] == 32
    assert p.pool[1] == 4


def test_block_ids_out_of_range_give_no_slot(pkv):
    p = Pool(2, 4, 8, 0, 8, 4, 8)
    p.ring[1] = 99
    p.dev["ring"][1] = 99
    slots, err = p.step(pkv, [8, 3], 20)
    assert err == 1 and (slots[4:8] == -1).all() and (slots[8:11] >= 0).all()


def test_largest_table(pkv):
    """One request growing by a long prompt, and the sums' 32-bit edge: more tokens wanted than
    rows can name are refused."""
    MB, bs = 40000, 16
    p = Pool(1, MB, MB, 17, MB, bs, MB)
    p.step(pkv, [600001], 600010)
    p.step(pkv, [600002], 1)
    p.step(pkv, [123], 0)
    q = Pool(70, 4, 8, 0, 8, 2**25, 8)
    slots, err = q.step(pkv, [2**27] * 70, 5)
    assert err == 32 and (q.lens == 0).all()


def test_graph_replays_and_streams(pkv):
    """A captured step replayed: the lengths and the pool move on with each replay; a second
    graph on the same pool alternates with it."""
    B, bs, MB = 40, 16, 8
    p = Pool(B, MB, B * MB, 5, B * MB, bs, B * MB)
    p.step(pkv, np.arange(B), int(np.arange(B).sum()))
    target = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.empty(B, dtype=torch.int64, device="cuda")
    start = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    graphs = []
    side = torch.cuda.Stream()
    for delta in (1, -2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            torch.add(p.dev["lens"], delta, out=target)
            target.clamp_(min=0)
            pkv.kv_resize_requests(p.dev["tables"], p.dev["lens"], target, p.dev["ring"],
                                   p.dev["pool"], slots, start, bs, p.num_blocks)
        graphs.append((g, delta))
    for i in (0, 0, 1, 0, 1, 0, 0):
        g, delta = graphs[i]
        g.replay()
        want, want_start, err = ref.resize(p.tables, p.lens, np.maximum(p.lens + delta, 0), p.ring,
                                           p.pool, B, bs, p.num_blocks)
        assert pkv.pkv_device_error() == err == 0
        assert np.array_equal(slots.cpu().numpy(), want)
        for k in ("ring", "pool", "tables", "lens"):
            assert np.array_equal(p.dev[k].cpu().numpy(), getattr(p, k)), k
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        p.step(pkv, p.lens + 3, 3 * B)


def test_many_rows_in_a_graph(pkv):
    """More rows than one cluster takes: the two grids of that form, captured and replayed."""
    B, bs, MB, rows = 300, 16, 40, 20000
    p = Pool(B, MB, B * MB, 9, B * MB, bs, B * MB)
    p.step(pkv, np.arange(B), rows)
    target = torch.zeros(B, dtype=torch.int32, device="cuda")
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    start = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pkv.kv_resize_requests(p.dev["tables"], p.dev["lens"], target, p.dev["ring"],
                               p.dev["pool"], slots, start, bs, p.num_blocks)
    for delta in (60, -7, 70, 66, -500):  # 66: more than the rows
        want_target = np.maximum(p.lens + delta, 0).astype(np.int32)
        target.copy_(torch.from_numpy(want_target))
        g.replay()
        want, want_start, err = ref.resize(p.tables, p.lens, want_target, p.ring, p.pool, rows, bs,
                                           p.num_blocks)
        assert pkv.pkv_device_error() == err
        assert np.array_equal(slots.cpu().numpy(), want)
        assert np.array_equal(start.cpu().numpy(), want_start)
        for k in ("ring", "pool", "tables", "lens"):
            assert np.array_equal(p.dev[k].cpu().numpy(), getattr(p, k)), k
