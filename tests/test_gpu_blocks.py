"""pkv_kv_blocks_update against block tables and a stack in plain lists: every
value is a whole number, so everything must be equal."""
import numpy as np
import pytest
import torch

from paged_kv_cache_41_gb300 import pkv

from step_util import Blocks

pytestmark = pytest.mark.gpu
I32 = torch.int32


class Step:
    """Requests of given lengths over a pool, on the GPU and as the plain form."""

    def __init__(self, lens, width, p=16, spare=50, seed=0, nb=None):
        rng = np.random.default_rng(seed)
        self.p, need = p, [-(-int(t) // p) for t in lens]
        self.nb = nb or sum(need) + spare
        ids = rng.permutation(self.nb).astype(np.int32)
        tables = np.full((len(lens), width), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            tables[r, :n] = ids[at:at + n]
            at += n
        free = np.concatenate([ids[at:], ids[:at]])
        self.plain = Blocks(self.nb, p, tables, free, self.nb - at)
        self.lens_np = np.array(lens, np.int32)
        self.pool = torch.empty(self.nb, p, 1, 8, dtype=torch.bfloat16, device="cuda")
        self.tables, self.free = torch.from_numpy(tables).cuda(), torch.from_numpy(free).cuda()
        self.count = torch.tensor([self.nb - at], dtype=I32, device="cuda")
        self.lens = torch.from_numpy(self.lens_np).cuda()

    def put(self):
        """The plain form's tables, stack and count to the GPU (after a test changed them)."""
        self.tables.copy_(torch.tensor(self.plain.tables, dtype=I32))
        self.free.copy_(torch.tensor(self.plain.free, dtype=I32))
        self.count.fill_(self.plain.count)

    def update(self, base, add, num_rows, window=0, sinks=0, **kw):
        """One call on both, compared; base: "lens", None or lengths."""
        base_np = self.lens_np if isinstance(base, str) else None if base is None else np.array(base, np.int32)
        want = self.plain.update(self.lens_np, base_np, add, num_rows, window, sinks)
        base_t = self.lens if isinstance(base, str) else None if base is None else torch.from_numpy(base_np).cuda()
        got = pkv.kv_blocks_update(self.pool, self.tables, self.lens,
                                   torch.tensor(np.array(add, np.int64), device="cuda").to(I32), self.free,
                                   self.count, base_lens=base_t, num_rows=num_rows, window=window,
                                   num_sinks=sinks, **kw)
        err = pkv.get_device_error()
        assert err == self.plain.err
        self.plain.err = 0
        for name, g, w in zip(("out_lens", "row_ptr", "slots", "positions"), got, want):
            assert g.tolist() == w, name
        self.same()
        self.lens, self.lens_np = got[0], np.array(want[0], np.int32)
        return got, err

    def same(self):
        assert self.tables.cpu().tolist() == self.plain.tables
        assert self.free.cpu().tolist() == self.plain.free
        assert self.count.item() == self.plain.count


@pytest.mark.parametrize("p", [1, 7, 16, 64, 256])
@pytest.mark.parametrize("batch", [1, 3, 64])
def test_random_steps(p, batch):
    rng = np.random.default_rng(p * 100 + batch)
    width = 12
    s = Step(rng.integers(0, 6 * p + 1, batch), width, p, spare=batch * 8, seed=p)
    for k in range(12):
        kind = k % 4
        if kind == 0:    # one row each, some none
            add = rng.integers(0, 2, batch)
            s.update("lens", add, int(add.sum()))
        elif kind == 1:  # drafts, then those that were accepted
            old, add = s.lens_np.copy(), rng.integers(0, 2 * p + 1, batch)
            add = np.minimum(add, width * p - old)
            (lens, _, _, _), err = s.update("lens", add, int(add.sum()) + 5)
            s.update(old, np.minimum(rng.integers(0, 2 * p + 1, batch), s.lens_np - old), 0)
        elif kind == 2:  # an eviction, a request that ends, one that starts
            add = np.minimum(s.lens_np, rng.integers(0, 4 * p + 1, batch))
            s.update(None, add, 0)
        else:
            add = np.where(s.lens_np == 0, rng.integers(0, 5 * p + 1, batch), s.lens_np)
            s.update(None, add, int(np.maximum(add - s.lens_np, 0).sum()))


def test_a_growth_and_its_undoing_leave_everything_as_it_was():
    s = Step([5, 100, 0, 64, 31], 20, spare=40)
    tables, free, count = s.tables.clone(), s.free.clone(), s.count.clone()
    old = s.lens_np.copy()
    s.update("lens", [60, 0, 17, 100, 1], 178)
    assert not torch.equal(tables, s.tables)
    s.update(old, [0] * 5, 0)
    assert torch.equal(tables, s.tables) and torch.equal(free, s.free) and torch.equal(count, s.count)


@pytest.mark.parametrize("batch", [1023, 1024, 1025, 2500])
def test_more_requests_than_threads(batch):
    rng = np.random.default_rng(batch)
    s = Step(rng.integers(0, 100, batch), 16, spare=3000, seed=1)
    add = rng.integers(0, 40, batch)
    s.update("lens", add, int(add.sum()) + 9)     # past the rows the one CTA writes itself
    s.update(None, np.minimum(s.lens_np, rng.integers(0, 60, batch)), 0)
    add = rng.integers(0, 2, batch)
    s.update("lens", add, int(add.sum()))


def test_65535_requests():
    s = Step(np.arange(65535) % 3, 2, p=2, spare=200000)
    s.update("lens", np.arange(65535) % 2, 40000)
    s.update(None, (s.lens_np + 1) // 2, 10)


def test_long_requests():
    s = Step([65536, 3, 40000], 70000 // 16 + 1, spare=5000)
    s.update("lens", [1, 65533, 20000], 90000)
    s.update(None, [0, 65536, 7], 0)
    s.update("lens", [70000, 0, 5], 70005)


def test_rows_around_what_one_cta_writes():
    for rows in (4095, 4096, 4097):
        s = Step([10, 20], 300, spare=300)
        s.update("lens", [4000, rows - 4000], rows)


@pytest.mark.parametrize("rows", [0, 1, 5000])
def test_no_requests(rows):
    got = pkv.kv_blocks_update(torch.empty(4, 16, 1, 8, device="cuda", dtype=torch.bfloat16),
                               torch.empty(0, 3, dtype=I32, device="cuda"), torch.empty(0, dtype=I32, device="cuda"),
                               torch.empty(0, dtype=I32, device="cuda"), torch.zeros(4, dtype=I32, device="cuda"),
                               torch.tensor([3], dtype=I32, device="cuda"), num_rows=rows)
    assert got[1].tolist() == [0] and (got[2] == -1).all() and (got[3] == -1).all()


# ------------------------------------------------------------------ refusals
def test_exhaustion_serves_in_order():
    # 5 blocks left: the second takes 3, the third lacks one, the fourth needs none
    s = Step([16, 16, 16, 10, 16], 20, spare=5)
    got, err = s.update("lens", [0, 48, 48, 3, 1], 100)
    assert err == pkv.DEVERR_POOL
    assert got[0].tolist() == [16, 64, 16, 13, 16] and s.count.item() == 2
    # what is given back in the same call can be taken
    s.update(None, [0, 0, 64, 13, 48], 100)


def test_lengths_that_make_no_sense():
    s = Step([5, 33, 16, 8, 8], 4, spare=30)
    got, err = s.update("lens", [-6, 40, 0, 1, 2**31 - 1], 50)
    assert err == pkv.DEVERR_LENGTH
    assert got[0].tolist() == [5, 33, 16, 9, 8]
    s.update([-1, 70, 0, 0, 5], [3, -70, 2**31 - 1, 65, -5], 50)
    s.lens_np = np.array([-3, 65, 16, 70, 0], np.int32)
    s.lens = torch.from_numpy(s.lens_np).cuda()
    s.update("lens", [4, 0, 1, -69, 1], 50)


def test_rows_that_pass_the_step():
    s = Step([0, 0, 0, 0], 4, spare=30)
    got, err = s.update("lens", [10, 20, 5, 0], 25)
    assert err == pkv.DEVERR_LENGTH
    assert got[0].tolist() == [10, 0, 0, 0] and got[1].tolist() == [0, 10, 25, 25, 25]


def test_bad_ids():
    s = Step([40, 40, 40], 8, spare=10)
    s.plain.tables[1][2] = s.nb        # given back: dropped
    s.plain.tables[2][1] = -1          # nothing to give back
    top = s.plain.count - 1
    s.plain.free[top - 1] = -7         # taken: -1
    s.plain.free[top - 2] = 2**31 - 1
    s.put()
    _, err = s.update("lens", [60, 0, 0], 60)
    assert err == pkv.DEVERR_BLOCK
    _, err = s.update(None, [40, 0, 0], 0)
    assert err == pkv.DEVERR_BLOCK


@pytest.mark.parametrize("count", [-1, 10**6])
def test_bad_counts(count):
    s = Step([40, 40], 8, spare=10)
    s.plain.count = count
    s.put()
    s.update("lens", [1, 30], 31)


def test_an_id_given_back_twice_stays_inside_the_stack():
    s = Step([64, 64], 8, spare=0)
    s.plain.tables[1] = list(s.plain.tables[0])   # two requests with the same blocks
    s.plain.count = s.nb - 6
    s.put()
    _, err = s.update(None, [0, 0], 0)
    assert err == pkv.DEVERR_BLOCK and s.count.item() == s.nb


# -------------------------------------------------------------- the window
@pytest.mark.parametrize("p,window,sinks", [(16, 1, 0), (16, 16, 0), (16, 17, 1), (16, 100, 40), (4, 7, 5),
                                            (64, 64, 64), (1, 3, 2)])
def test_window_gives_back_what_lies_behind_it(p, window, sinks):
    rng = np.random.default_rng(window)
    batch = 40
    s = Step(rng.integers(0, 20 * p, batch), 64, p, spare=batch * 12, seed=2)
    for k in range(3 * p if p < 16 else 20):
        add = rng.integers(0, 3, batch)
        s.update("lens", add, int(add.sum()), window, sinks)
        for r, t in enumerate(s.lens_np):
            seen = {x // p for x in range(t) if x < sinks or x >= t - window}
            assert all(s.plain.tables[r][j] >= 0 for j in seen)
    s.update(None, [0] * batch, 0, window, sinks)
    assert s.count.item() == s.nb


def test_window_over_a_long_prompt():
    s = Step([0, 5000, 70000], 5000, spare=6000)
    s.update("lens", [20000, 1, 1], 20002, 1000, 4)     # nothing of a prompt goes while it is read
    assert (s.tables[0, :1250] >= 0).all()
    s.update("lens", [1, 1, 1], 3, 1000, 4)
    assert (s.tables[0, 1:1187] == -1).all() and s.tables[0, 0] >= 0


# ----------------------------------------------------------- graphs, streams
def test_graph_replays_and_two_at_once():
    steps = [Step([5, 17, 32, 0], 64, spare=200, seed=k) for k in range(2)]
    graphs, bufs = [], []
    for s in steps:
        other = s.lens.clone()
        add = torch.tensor([1, 2, 0, 3], dtype=I32, device="cuda")
        out = [torch.empty(4, dtype=I32, device="cuda"), torch.empty(5, dtype=I32, device="cuda"),
               torch.empty(8, dtype=torch.int64, device="cuda"), torch.empty(8, dtype=I32, device="cuda")]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                pkv.kv_blocks_update(s.pool, s.tables, other, add, s.free, s.count, base_lens=other,
                                     out_lens=out[0], row_ptr=out[1], slots=out[2], positions=out[3])
                other.copy_(out[0])
        graphs.append(g)
        bufs.append((other, out, add))  # a graph keeps none of them alive
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for k in range(9):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for s, (_, out, _) in zip(steps, bufs):
            want = s.plain.update(s.lens_np, s.lens_np, [1, 2, 0, 3], 8)
            for g_, w in zip(out, want):
                assert g_.tolist() == w
            s.lens_np = np.array(want[0], np.int32)
            s.same()
    assert pkv.get_device_error() == 0


def test_side_stream():
    s = Step([5, 17], 64, spare=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    add = torch.tensor([40, 1], dtype=I32, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    got = pkv.kv_blocks_update(s.pool, s.tables, s.lens, add, s.free, s.count, base_lens=s.lens, num_rows=41,
                               stream=side)
    side.synchronize()
    want = s.plain.update(s.lens_np, s.lens_np, [40, 1], 41)
    for g, w in zip(got, want):
        assert g.tolist() == w
    s.same()


def test_slots_are_those_that_the_append_takes():
    # a prompt appended through the slots, read back through the table
    s = Step([0, 0], 8, p=16, spare=16)
    got, _ = s.update("lens", [50, 20], 72)
    kc = torch.zeros(s.nb, 16, 1, 64, dtype=torch.float32, device="cuda")
    rows = torch.randn(72, 1, 64, device="cuda")
    pkv.kv_append(kc, kc.clone(), rows, rows, got[2])
    for r, (a, n) in enumerate(((0, 50), (50, 20))):
        flat = kc[s.tables[r, : -(-n // 16)].long()].view(-1, 64)[:n]
        assert torch.equal(flat, rows[a:a + n, 0])
    assert pkv.get_device_error() == 0
