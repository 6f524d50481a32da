"""The page table on the GPU against a list-based model of it: pages, slots,
positions, lengths and the free stack are whole numbers and have to be equal."""
import random

import pytest
import torch

import hybrid_ssm_decode_gb300 as rssm

pytestmark = pytest.mark.gpu


class Model:
    """The page table in Python lists (include/rssm.h, "page table")."""

    def __init__(self, batch, ps, num, most, free):
        self.B, self.ps, self.num, self.most = batch, ps, num, most
        self.free = list(free)                       # the stack; the last entry is its top
        self.rows = [[] for _ in range(batch)]
        self.lens = [0] * batch

    def extend(self, new, max_tokens):
        need, off = [], 0
        for b, n in enumerate(new):
            ok = n >= 0 and self.lens[b] + n <= self.most * self.ps
            off += max(n, 0)
            ok = ok and off <= max_tokens
            need.append(-(-(self.lens[b] + n) // self.ps) - len(self.rows[b]) if ok else None)
        run, served = 0, []
        for w in need:                               # the scan stops at the first that does not fit
            if w is None:
                served.append(False)
                continue
            run += w
            served.append(w == 0 or run <= len(self.free))
        total = sum(w for w, s in zip(need, served) if s)
        pages = self.free[len(self.free) - total:] if total else []
        self.free = self.free[:len(self.free) - total]
        slots, pos, at = [], [], 0
        for b, n in enumerate(new):
            n0 = max(n, 0)
            if not served[b]:
                slots += [-1] * n0
                pos += [-1] * n0
                continue
            self.rows[b] += pages[at:at + need[b]]
            at += need[b]
            for i in range(self.lens[b], self.lens[b] + n):
                slots.append(self.rows[b][i // self.ps] * self.ps + i % self.ps)
                pos.append(i)
            self.lens[b] += n
        return slots[:max_tokens], pos[:max_tokens], served

    def cut(self, newlens):
        for b, n in enumerate(newlens):
            left = -(-n // self.ps)
            self.free += self.rows[b][left:]
            self.rows[b] = self.rows[b][:left]
            self.lens[b] = n

    def check(self, pt):
        torch.cuda.synchronize()
        assert pt.lens.tolist() == self.lens
        n = int(pt.free_count)
        assert n == len(self.free)
        lay = pt.layout
        stack = pt.workspace[lay.free:lay.free + 4 * self.num].view(torch.int32).tolist()
        assert stack[:n] == self.free
        want = torch.full((self.B, self.most), -1, dtype=torch.int32)
        for b, r in enumerate(self.rows):
            want[b, :len(r)] = torch.tensor(r, dtype=torch.int32)
        assert torch.equal(pt.table.cpu(), want)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("batch,ps,num,most", [
    (1, 16, 5, 3), (3, 1, 40, 20), (64, 16, 900, 40), (257, 7, 3000, 30), (1024, 16, 5000, 9), (1025, 32, 2500, 5),
    (3000, 16, 9000, 6)])
def test_random_walk_matches_model(cuda_lib, batch, ps, num, most):
    """Extends (uniform and ragged), rollbacks and truncations in turn, from a
    shuffled free stack; the pool runs out now and then."""
    rng = random.Random(batch * 31 + ps)
    order = list(range(num))
    rng.shuffle(order)
    pt = rssm.PageTable(batch, ps, num, most, free=_i32(order))
    m = Model(batch, ps, num, most, order)
    m.check(pt)
    for step in range(12):
        kind = rng.choice(["uniform", "ragged", "ragged", "truncate"])
        if kind == "truncate":
            keep = [rng.choice([0, rng.randint(0, most * ps + 5), m.lens[b]]) for b in range(batch)]
            pt.truncate(_i32(keep))
            m.cut([min(n, k) for n, k in zip(m.lens, keep)])
        else:
            T = rng.randint(1, 8)
            new = [T] * batch if kind == "uniform" else [rng.choice([0, 1, rng.randint(0, 2 * ps + 1)]) for _ in range(batch)]
            total = sum(new)
            slots = torch.full((total + 5,), -7, dtype=torch.int32, device="cuda")
            pos = torch.full((total + 5,), -7, dtype=torch.int32, device="cuda")
            if kind == "uniform":
                pt.extend(slots, T=T, positions=pos)
            else:
                pt.extend(slots, new=_i32(new), positions=pos)
            s, p, served = m.extend(new, total + 5)
            assert slots.tolist() == s + [-7] * 5 and pos.tolist() == p + [-7] * 5
            err = pt.get_error()
            assert (err[0] == 0) == all(served) and err[1] == served.count(False)
            if kind == "uniform" and all(served):
                acc = [rng.randint(0, T) for _ in range(batch)]
                pt.rollback(T, _i32(acc))
                m.cut([n - T + a for n, a in zip(m.lens, acc)])
        m.check(pt)
    assert pt.get_error()[0] == 0


@pytest.mark.parametrize("offset", [0, 1])
def test_many_blocks_and_unaligned_lists(cuda_lib, offset):
    """Prompts of several hundred thousand tokens, with lists that do and do
    not start on 16 bytes, and back again."""
    batch, ps, most = 300, 16, 1000
    rng = random.Random(5)
    new = [rng.randint(0, most * ps) for _ in range(batch)]
    num = sum(-(-n // ps) for n in new)              # every page goes out
    pt = rssm.PageTable(batch, ps, num, most)
    m = Model(batch, ps, num, most, range(num))
    slots = torch.empty(sum(new) + offset, dtype=torch.int32, device="cuda")[offset:]
    pos = torch.empty(sum(new) + offset, dtype=torch.int32, device="cuda")[offset:]
    for _ in range(2):
        pt.extend(slots, new=_i32(new), positions=pos)
        s, p, served = m.extend(new, sum(new))
        assert all(served)
        assert slots.tolist() == s and pos.tolist() == p
        m.check(pt)
        pt.truncate(_i32([0] * batch))
        m.cut([0] * batch)
        m.check(pt)


@pytest.mark.parametrize("batch,T,ps", [(9000, 3, 16), (9000, 6, 16), (40, 17, 16), (40, 300, 1), (1500, 16, 5), (300, 13, 4)])
def test_uniform_steps_of_either_kind(cuda_lib, batch, T, ps):
    """Uniform extends and rollbacks past the single-block kernels' batch and tokens, and below."""
    most = 2 + 2 * T // ps
    num = batch * (1 + 2 * T // ps) - 3              # the last requests of the second round get none
    order = list(range(num))
    random.Random(1).shuffle(order)
    pt, m = rssm.PageTable(batch, ps, num, most, free=_i32(order)), Model(batch, ps, num, most, order)
    slots, pos = (torch.empty(batch * T, dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(3):
        pt.extend(slots, T=T, positions=pos)
        s, p, served = m.extend([T] * batch, batch * T)
        assert slots.tolist() == s and pos.tolist() == p
        err = pt.get_error()
        assert (err[0] == 0) == all(served) and err[1] == served.count(False)
        m.check(pt)
        if step == 1:
            acc = [(b * 7) % (T + 1) if served[b] else T for b in range(batch)]
            pt.rollback(T, _i32(acc))
            short = [n < T for n in m.lens]          # never served: refused, and unchanged
            assert pt.get_error()[1] == sum(short)
            m.cut([n if x else n - T + a for n, a, x in zip(m.lens, acc, short)])
            m.check(pt)
    assert pt.get_error()[0] == 0


def test_a_rejected_draft_round_leaves_no_trace(cuda_lib):
    batch, ps = 100, 16
    pt = rssm.PageTable(batch, ps, 500, 8)
    slots = torch.empty(batch * 8, dtype=torch.int32, device="cuda")
    pt.extend(torch.empty(5000, dtype=torch.int32, device="cuda"), new=_i32([i % 40 for i in range(batch)]))
    torch.cuda.synchronize()
    before = pt.workspace.clone()
    pt.extend(slots, T=8)
    assert not torch.equal(pt.workspace, before)
    pt.rollback(8, _i32([0] * batch))
    torch.cuda.synchronize()
    assert torch.equal(pt.workspace, before)


def test_refused_requests_stay_as_they_were(cuda_lib):
    pt = rssm.PageTable(4, 16, 6, 2)                 # rows of 32 tokens, 6 pages
    m = Model(4, 16, 6, 2, range(6))

    def go(new, max_tokens=200):
        slots = torch.full((max_tokens,), -7, dtype=torch.int32, device="cuda")
        pt.extend(slots, new=_i32(new))
        s, _, served = m.extend(new, max_tokens)
        assert slots.tolist()[:len(s)] == s
        m.check(pt)
        return pt.get_error(), served

    err, served = go([16, 33, 1, 1])                 # the second passes its row
    assert served == [True, False, True, True] and err == (rssm.RSSM_DEV_PAGES_ROW, 1, 1, 33)
    err, served = go([16, -2, 0, 0])                 # a negative count
    assert served == [True, False, True, True] and err == (rssm.RSSM_DEV_PAGES_COUNT, 1, 1, -2)
    err, served = go([0, 20, 15, 20])                # 2 pages left: the second takes both, the last gets none
    assert served == [True, True, True, False] and err == (rssm.RSSM_DEV_PAGES_EMPTY, 1, 3, 20)
    pt.truncate(_i32([0, 99, 99, 99]))
    m.cut([0] + m.lens[1:])
    err, served = go([3, 4, 0, 5], max_tokens=8)     # slots for the first two only
    assert served == [True, True, True, False] and err == (rssm.RSSM_DEV_PAGES_SLOTS, 1, 3, 5)
    before = (pt.lens.tolist(), pt.table.tolist())
    pt.rollback(2, _i32([3, -1, 0, 2]))              # out of 0..2, twice; a request shorter than the drafts
    e = pt.get_error()
    assert e[0] == rssm.RSSM_DEV_PAGES_COUNT and e[1] == 3
    m.cut([m.lens[0], m.lens[1], m.lens[2] - 2, m.lens[3]])
    m.check(pt)
    pt.truncate(_i32([-1, 2 ** 31 - 1, 99, 99]))
    assert pt.get_error()[:3] == (rssm.RSSM_DEV_PAGES_COUNT, 1, 0)
    assert before[0][0] == pt.lens.tolist()[0]
    m.check(pt)


@pytest.mark.parametrize("batch,T,ragged", [(3, 4, False), (3, 4, True), (3, 40, False), (1500, 3, False), (1500, 3, True),
                                            (1500, 20, False), (1100, 6, False)])
def test_a_refused_request_is_not_rolled_back(cuda_lib, batch, T, ragged):
    """The pool gives out in the middle of a batch: a rollback of the whole round
    leaves every request as it was before, the refused ones with all their tokens."""
    ps = 4
    lens = [T + b % 5 for b in range(batch)]
    held = [-(-n // ps) for n in lens]
    need = [-(-(n + T) // ps) - h for n, h in zip(lens, held)]
    late = [need[b] > 0 and b > batch // 2 for b in range(batch)]
    num = sum(held) + sum(need[:batch // 2 + 1])
    pt = rssm.PageTable(batch, ps, num, 2 + 3 * T // ps)
    slots = torch.empty(sum(lens) + batch * T, dtype=torch.int32, device="cuda")

    def state():
        return pt.lens.tolist(), pt.table.tolist(), pt.free_count.tolist()

    def go():
        pt.extend(slots, **(dict(new=_i32([T] * batch)) if ragged else dict(T=T)))

    pt.extend(slots, new=_i32(lens))
    before = state()
    go()
    assert pt.refused.tolist() == [int(x) for x in late]
    assert pt.get_error()[:2] == (rssm.RSSM_DEV_PAGES_EMPTY, sum(late))
    pt.extend(slots, new=_i32([0] * batch))          # asks for nothing: changes nothing
    pt.rollback(T, _i32([0] * batch))
    assert state() == before and pt.get_error()[0] == 0
    # drafts that stay, and room for the late ones once the first request has left
    go()
    pt.rollback(T, _i32([b % (T + 1) for b in range(batch)]))
    assert pt.lens.tolist() == [n if x else n + b % (T + 1) for b, (n, x) in enumerate(zip(lens, late))]
    pt.truncate(_i32([0 if b <= batch // 2 else 10 ** 6 for b in range(batch)]))
    pt.get_error()
    go()
    assert not any(pt.refused.tolist()) and pt.get_error()[0] == 0
    grown = pt.lens.tolist()
    pt.rollback(T, _i32([1] * batch))
    assert pt.lens.tolist() == [n - T + 1 for n in grown]


def test_refusals_of_each_kind_are_marked(cuda_lib):
    pt = rssm.PageTable(4, 16, 6, 2)
    slots = torch.empty(64, dtype=torch.int32, device="cuda")
    pt.extend(slots, new=_i32([16, 16, 1, 1]))
    pt.extend(slots, new=_i32([0, 17, -1, 0]))       # past its row; a negative count
    assert pt.refused.tolist() == [0, 1, 1, 0]
    pt.extend(slots[:4], new=_i32([0, 0, 4, 1]))     # slots for the third alone
    assert pt.refused.tolist() == [0, 1, 0, 1]
    pt.rollback(1, _i32([0, 0, 0, 0]))
    assert pt.lens.tolist() == [15, 16, 4, 1]


def test_extend_by_nothing(cuda_lib):
    """No slots, and counts that are all 0."""
    pt = rssm.PageTable(4, 16, 8, 2)
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    pt.extend(none, new=_i32([0, 0, 0, 0]), positions=none)
    assert pt.get_error()[0] == 0 and pt.lens.tolist() == [0] * 4


def test_a_request_that_asks_for_nothing_is_not_refused(cuda_lib):
    """Behind requests that the slot list cannot hold, and an empty pool."""
    pt = rssm.PageTable(4, 16, 2, 2)
    slots = torch.empty(3, dtype=torch.int32, device="cuda")
    pt.extend(slots, new=_i32([2, 2, 0, 1]))
    assert pt.get_error()[:2] == (rssm.RSSM_DEV_PAGES_SLOTS, 2)
    assert pt.refused.tolist() == [0, 1, 0, 1] and pt.lens.tolist() == [2, 0, 0, 0]
    pt.extend(torch.empty(0, dtype=torch.int32, device="cuda"), new=_i32([0, 1, 0, 1]))
    assert pt.get_error()[:2] == (rssm.RSSM_DEV_PAGES_SLOTS, 2)
    pt.extend(torch.empty(40, dtype=torch.int32, device="cuda"), new=_i32([0, 16, 0, 16]))
    assert pt.get_error() == (rssm.RSSM_DEV_PAGES_EMPTY, 1, 3, 16)
    assert pt.refused.tolist() == [0, 0, 0, 1] and pt.lens.tolist() == [2, 16, 0, 0]


def test_binding_refuses(cuda_lib):
    pt = rssm.PageTable(4, 16, 8, 2)
    good = torch.empty(8, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        pt.extend(good.long(), T=1)
    with pytest.raises(ValueError):
        pt.extend(good.cpu(), T=1)
    with pytest.raises(ValueError):
        pt.extend(good[::2], T=1)
    with pytest.raises(ValueError):
        pt.extend(good)
    with pytest.raises(ValueError):
        pt.extend(good, T=1, new=good[:4])
    with pytest.raises(ValueError):
        pt.extend(good, new=good[:3])
    with pytest.raises(ValueError):
        pt.rollback(1, good)
    with pytest.raises(rssm.RssmError):
        pt.extend(good[:3], T=1)                     # four tokens, three slots
    with pytest.raises(rssm.RssmError):
        pt.rollback(0, good[:4])
    with pytest.raises(rssm.RssmError):
        rssm.PageTable(4, 16, 2 ** 28, 2)            # slots past 31 bits
    pt.close()
