"""Shortening a sequence of the host pool: the end of an eviction and of a
speculative step."""
import numpy as np
import pytest

from paged_kv_cache_41_gb300.pool import BlockPool


@pytest.mark.parametrize("p", [1, 4, 16])
@pytest.mark.parametrize("length", [0, 1, 4, 5, 16, 17, 31, 32, 33, 40])
def test_blocks_past_the_new_length_are_free(p, length):
    pool = BlockPool(64, p, seed=1)
    s = pool.new_seq()
    s.append(40)
    ids = s.blocks()
    s.truncate(length)
    keep = -(-length // p)
    assert s.length == length and s.num_blocks == keep and np.array_equal(s.blocks(), ids[:keep])
    assert pool.num_free == 64 - keep
    assert [pool.refcount(int(b)) for b in ids] == [1] * keep + [0] * (len(ids) - keep)
    # the next tokens go to positions length, length + 1, ...
    slots, cow = s.append(7)
    table = s.blocks().astype(np.int64)
    pos = length + np.arange(7)
    assert np.array_equal(slots, table[pos // p] * p + pos % p) and len(cow) == 0
    s.release()
    assert pool.num_free == 64


def test_shared_blocks_lose_one_reference_and_the_tail_is_copied_on_write():
    pool = BlockPool(32, 16, seed=2)
    s = pool.new_seq()
    s.append(50)
    kid = s.fork()
    ids = s.blocks()
    s.truncate(20)
    assert [pool.refcount(int(b)) for b in ids] == [2, 2, 1, 1]
    assert kid.length == 50 and np.array_equal(kid.blocks(), ids)
    slots, cow = s.append(1)  # its tail holds rows of the child
    assert len(cow) == 1 and cow[0, 0] == ids[1] and slots[0] == cow[0, 1] * 16 + 4
    kid.release()
    s.release()
    assert pool.num_free == 32


def test_lengths_outside_the_sequence_are_refused():
    pool = BlockPool(8, 16)
    s = pool.new_seq()
    s.append(30)
    for bad in (-1, 31, 2**40):
        with pytest.raises(ValueError):
            s.truncate(bad)
    assert s.length == 30 and pool.num_free == 6
    s.truncate(30)
    assert s.length == 30 and s.num_blocks == 2
    s.release()


def test_speculation_and_eviction_keep_the_pool_whole():
    rng = np.random.default_rng(3)
    pool = BlockPool(64, 16, seed=4)
    seqs = [pool.new_seq() for _ in range(3)]
    lens = [0, 0, 0]
    for step in range(300):
        i = int(rng.integers(0, 3))
        drafted = int(rng.integers(1, 20))
        seqs[i].append(drafted)
        lens[i] += int(rng.integers(0, drafted + 1))  # the accepted ones
        seqs[i].truncate(lens[i])
        if lens[i] > 200:  # over the budget
            lens[i] = 96
            seqs[i].truncate(96)
        tables, got = pool.block_tables(seqs)
        assert got.tolist() == lens
        used = tables[tables >= 0]
        assert len(set(used.tolist())) == len(used) == sum(-(-t // 16) for t in lens)
        assert pool.num_free == 64 - len(used)
    for s in seqs:
        s.release()
    assert pool.num_free == 64
