"""Page bookkeeping against a model that serves one sequence at a time: tables,
lengths, counts and page contents equal; pools of every fill, odd sizes and
alignments; calls that cannot be served change nothing."""
import numpy as np
import pytest
import torch

import w8a8_quantized_projections_gb300 as clef
from decode_util import Pages, dev_i32

pytestmark = pytest.mark.gpu


class Pool:
    def __init__(self, rng, pages, seqs, width, page=16, heads=1, dim=64, planes=4, offset=0):
        self.P = page
        self.codes = torch.from_numpy(rng.integers(0, 256, (planes, pages, heads, page, dim), dtype=np.uint8)).cuda()
        self.scales = torch.from_numpy(rng.random((planes, pages, heads), dtype=np.float32)).cuda()
        self.table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.refs = torch.zeros(pages + offset, dtype=torch.int32, device="cuda")[offset:]
        self.model = Pages(np.full((seqs, width), -1, np.int32), [0] * seqs, np.zeros(pages, np.int32), page)

    def same(self):
        assert self.lens.tolist() == self.model.lens
        assert self.refs.tolist() == self.model.refs.tolist()
        for b, x in enumerate(self.model.lens):
            n = -(-x // self.P)
            assert self.table[b, :n].tolist() == self.model.table[b, :n].tolist()

    def reserve(self, grow):
        ok = self.model.reserve(grow)
        clef.kv_reserve(self.table, self.lens, self.refs, dev_i32(grow), self.P)
        assert clef.poll_status() == (0 if ok else 6)
        self.same()
        return ok

    def fork(self, src, dst):
        moves = self.model.fork(src, dst)
        want, sc = self.codes.clone(), self.scales.clone()
        for a, z in moves or []:
            want[:, z], sc[:, z] = want[:, a], sc[:, a]
        clef.kv_fork(self.codes, self.scales, self.table, self.lens, self.refs, dev_i32(src), dev_i32(dst))
        assert clef.poll_status() == (6 if moves is None else 0)
        self.same()
        assert torch.equal(self.codes, want) and torch.equal(self.scales, sc)

    def free(self, seqs):
        self.model.free(seqs)
        clef.kv_free(self.table, self.lens, self.refs, dev_i32(seqs), self.P)
        assert clef.poll_status() == 0
        self.same()

    def compact(self, apart=False):
        before = (self.table.clone(), self.refs.clone())
        live, moves = self.model.compact()
        want, sc = self.codes.clone(), self.scales.clone()
        for a, z in moves:
            want[:, z], sc[:, z] = want[:, a], sc[:, a]
        if apart:
            t, r = torch.full_like(self.table, -7), torch.full_like(self.refs, -7)
            got = clef.kv_compact(self.codes, self.scales, self.table, self.lens, self.refs, t, r)
            assert torch.equal(self.table, before[0]) and torch.equal(self.refs, before[1])
            self.table, self.refs = t, r
        else:
            got = clef.kv_compact(self.codes, self.scales, self.table, self.lens, self.refs)
        assert got.item() == live and clef.poll_status() == 0
        self.same()
        assert torch.equal(self.codes, want) and torch.equal(self.scales, sc)


@pytest.mark.parametrize("pages,seqs,offset", [(7, 2, 0), (64, 5, 1), (257, 9, 3), (1000, 30, 2), (20011, 50, 0)])
def test_a_life(pages, seqs, offset):
    """Random reserves, forks, frees and compactions."""
    rng = np.random.default_rng(pages)
    width = max(4, 2 * pages // seqs)
    pool = Pool(rng, pages, seqs, width, planes=2, offset=offset)
    for step in range(24):
        kind = rng.integers(4)
        lens = pool.model.lens
        if kind <= 1:
            grow = [int(rng.integers(0, max(1, min(4 * pages // seqs * 16, width * 16 - x)) )) if rng.random() < 0.6 else 0
                    for x in lens]
            if rng.random() < 0.2:
                grow = [min(width * 16 - x, g * 9) for x, g in zip(lens, grow)]
            pool.reserve(grow)
        elif kind == 2:
            empty = [b for b, x in enumerate(lens) if x == 0]
            full = [b for b, x in enumerate(lens) if x]
            if empty and full:
                k = int(rng.integers(1, len(empty) + 1))
                dst = [int(d) for d in rng.permutation(empty)[:k]]
                pool.fork([int(full[rng.integers(len(full))]) for _ in dst], dst)
        else:
            pool.free([int(b) for b in rng.permutation(seqs)[: rng.integers(1, seqs + 1)]])
        if step % 5 == 4:
            pool.compact(apart=step % 2 == 0)
    pool.free(list(range(seqs)))
    assert not pool.refs.any()


@pytest.mark.parametrize("page,heads,dim", [(16, 1, 64), (32, 3, 64), (64, 2, 256), (128, 8, 128)])
def test_page_shapes(page, heads, dim):
    rng = np.random.default_rng(page)
    pool = Pool(rng, 24, 6, 4, page, heads, dim, planes=6)
    pool.reserve([2 * page, page + 1, 1, 0, 0, 0])
    pool.fork([0, 1, 1], [3, 4, 5])
    pool.free([0, 2, 4])
    pool.compact()
    pool.compact()              # nothing left to move


def test_exactly_enough_and_one_too_few():
    rng = np.random.default_rng(1)
    pool = Pool(rng, 10, 3, 10)
    assert pool.reserve([64, 48, 33])              # 4 + 3 + 3 pages: all of them
    assert not pool.reserve([0, 1, 0])             # the next needs one
    assert pool.reserve([0, 0, 15])                # room in the last page
    pool.free([1])
    assert pool.reserve([0, 32, 0])
    pool.free([0])
    pool.fork([1], [0])                            # no part-filled page: nothing is taken
    pool.fork([], [])


def test_many_sequences():
    """More sequences than a CTA has threads, and the most there may be."""
    for seqs in (1025, 4096):
        rng = np.random.default_rng(seqs)
        pool = Pool(rng, seqs + 5, seqs, 2, planes=1)
        grow = rng.integers(0, 17, seqs)
        ok = pool.model.reserve([0] * seqs)
        assert ok
        clef.kv_reserve(pool.table, pool.lens, pool.refs, dev_i32(grow), 16)
        n = int((grow > 0).sum())
        want = np.full(seqs, -1)
        want[grow > 0] = np.arange(n)
        assert np.array_equal(pool.table[:, 0].cpu().numpy(), want)
        assert int(pool.refs.sum()) == n and pool.lens.tolist() == grow.tolist()
        clef.kv_free(pool.table, pool.lens, pool.refs, dev_i32(np.arange(seqs)), 16)
        assert not pool.refs.any() and not pool.lens.any() and clef.poll_status() == 0


def test_copy_pages():
    rng = np.random.default_rng(3)
    pool = Pool(rng, 12, 1, 1, heads=3, planes=6)
    want, sc = pool.codes.clone(), pool.scales.clone()
    want[:, [7, 0]], sc[:, [7, 0]] = want[:, [3, 11]], sc[:, [3, 11]]
    clef.kv_copy_pages(pool.codes, pool.scales, dev_i32([3, 11]), dev_i32([7, 0]))
    assert torch.equal(pool.codes, want) and torch.equal(pool.scales, sc)
    # leading dimensions of layers, and planes a pitch apart
    wide = torch.zeros((4, 13, 3, 16, 64), dtype=torch.uint8, device="cuda")
    wide[:, :12] = pool.codes[:4]
    wsc = pool.scales[:4].contiguous()
    clef.kv_copy_pages(wide[:, :12], wsc, dev_i32([1]), dev_i32([2]))
    assert torch.equal(wide[:, 2], pool.codes[:4, 1]) and not wide[:, 12].any()
    layers = pool.codes.view(3, 2, 12, 3, 16, 64)
    clef.kv_copy_pages(layers, pool.scales.view(3, 2, 12, 3), dev_i32([4]), dev_i32([5]))
    assert torch.equal(layers[:, :, 5], layers[:, :, 4])
    before = pool.codes.clone()
    clef.kv_copy_pages(pool.codes, pool.scales, dev_i32([0, 12, -3]), dev_i32([12, 0, 1]))
    assert clef.poll_status() == 5 and torch.equal(pool.codes, before)


def test_device_arguments_out_of_range_change_nothing():
    rng = np.random.default_rng(4)
    pool = Pool(rng, 20, 4, 3)
    pool.reserve([20, 16, 0, 0])
    state = lambda: (pool.table.clone(), pool.lens.clone(), pool.refs.clone(), pool.codes.clone())  # noqa: E731
    same = lambda a, b: all(torch.equal(x, y) for x, y in zip(a, b))                               # noqa: E731
    was = state()
    for grow in ([0, -1, 0, 0], [0, 0, 49, 0], [2 ** 31 - 1, 0, 0, 0]):
        clef.kv_reserve(pool.table, pool.lens, pool.refs, dev_i32(grow), 16)
        assert clef.poll_status() == 5 and same(was, state())
    for src, dst in (([0], [4]), ([-1], [2]), ([0], [1]), ([0, 1], [2, 2])):
        clef.kv_fork(pool.codes, pool.scales, pool.table, pool.lens, pool.refs, dev_i32(src), dev_i32(dst))
        assert clef.poll_status() == 5 and same(was, state()), (src, dst)
    pool.table[0, 1] = 20
    was = state()
    clef.kv_fork(pool.codes, pool.scales, pool.table, pool.lens, pool.refs, dev_i32([0]), dev_i32([2]))
    assert clef.poll_status() == 5 and same(was, state())
    pool.table[0, 1] = 1
    clef.kv_free(pool.table, pool.lens, pool.refs, dev_i32([9, -1]), 16)
    assert clef.poll_status() == 5 and torch.equal(pool.refs, was[2])
    clef.kv_free(pool.table, pool.lens, pool.refs, dev_i32([0, 0]), 16)      # listed twice: given back once
    assert clef.poll_status() == 0 and pool.refs.sum().item() == 1


def test_refusals():
    rng = np.random.default_rng(5)
    pool = Pool(rng, 8, 2, 2)
    t, n, r = pool.table, pool.lens, pool.refs
    for call in (lambda: clef.kv_reserve(t, n, r, dev_i32([1]), 16), lambda: clef.kv_reserve(t, n.long(), r, dev_i32([1, 1]), 16),
                 lambda: clef.kv_reserve(t.t(), n, r, dev_i32([1, 1]), 16),
                 lambda: clef.kv_fork(pool.codes, pool.scales, t, n, r[:7], dev_i32([0]), dev_i32([1])),
                 lambda: clef.kv_fork(pool.codes, pool.scales, t, n, r, dev_i32([0]), dev_i32([1, 0])),
                 lambda: clef.kv_compact(pool.codes, pool.scales, t, n, r, t[:, :1]),
                 lambda: clef.kv_copy_pages(pool.codes, pool.scales[:1], dev_i32([0]), dev_i32([1]))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: clef.kv_reserve(t, n, r, dev_i32([1, 1]), 20), lambda: clef.kv_free(t, n, r, dev_i32([0]), 0)):
        with pytest.raises(clef.ClefError):
            call()
    assert clef.poll_status() == 0


@pytest.mark.parametrize("order", ["before", "after"])
@pytest.mark.parametrize("pairs", [1, 40, 1300])
def test_fork_of_a_target(pairs, order):
    """A target that is a source too was empty before the call, so its copy is empty:
    no length, no page and no reference, wherever the two pairs stand in the list."""
    rng = np.random.default_rng(pairs)
    seqs = 1 + 2 * pairs
    pool = Pool(rng, pairs + 8, seqs, 3, planes=1)
    assert pool.reserve([37] + [0] * (seqs - 1))
    first, second = list(range(1, 1 + pairs)), list(range(1 + pairs, seqs))
    a, b = ([0] * pairs, first), (first, second)
    if order == "after":
        a, b = b, a
    clef.kv_fork(pool.codes, pool.scales, pool.table, pool.lens, pool.refs, dev_i32(a[0] + b[0]), dev_i32(a[1] + b[1]))
    assert clef.poll_status() == 0
    assert pool.lens.tolist() == [37] * (1 + pairs) + [0] * pairs
    assert (pool.table[second] == -1).all()
    refs = pool.refs.tolist()
    assert refs[:2] == [1 + pairs] * 2 and refs[2:3 + pairs] == [1] * (1 + pairs) and not any(refs[3 + pairs:])
    clef.kv_free(pool.table, pool.lens, pool.refs, dev_i32(list(range(seqs))), 16)
    assert clef.poll_status() == 0 and not pool.refs.any()


@pytest.mark.parametrize("seqs", [1, 5, 1025, 4096])
def test_rows_of_a_reservation(seqs):
    """The running sum of grow where it was served, zeros where it was not."""
    rng = np.random.default_rng(seqs)
    pool = Pool(rng, seqs + 1, seqs, 3, planes=1)
    rows = torch.full((seqs + 1,), -7, dtype=torch.int32, device="cuda")
    grow = rng.integers(0, 17, seqs)
    clef.kv_reserve(pool.table, pool.lens, pool.refs, dev_i32(grow), 16, row_start=rows)
    assert clef.poll_status() == 0 and rows.tolist() == [0] + np.cumsum(grow).tolist()
    was = pool.table.clone(), pool.lens.clone(), pool.refs.clone()
    for bad, status in (([32] * seqs, 6 if seqs > 1 else None), ([-1] + [0] * (seqs - 1), 5), ([49] + [1] * (seqs - 1), 5)):
        if status is None:
            continue
        rows.fill_(-7)
        clef.kv_reserve(pool.table, pool.lens, pool.refs, dev_i32(bad), 16, row_start=rows)
        assert clef.poll_status() == status and not rows.any()
        assert all(torch.equal(x, y) for x, y in zip(was, (pool.table, pool.lens, pool.refs)))
    for rows in (torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(seqs + 1, device="cuda")):
        with pytest.raises(ValueError):
            clef.kv_reserve(pool.table, pool.lens, pool.refs, dev_i32(grow), 16, row_start=rows)
