"""The table extension with a count of the blocks that each table holds: after
rejected drafts, and after the free list ran out, no block is lost or taken
twice.  Whole numbers: equal."""
import numpy as np
import pytest
import torch

from tests.test_gpu_cache_extend import owned
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu


def expected(table, held, seq, qsl, free, count, T, bs, D, I, d0, Dn):
    """(table, held, positions, slots, left, error) by the definition."""
    table, held, err = table.copy(), held.copy(), 0
    local = table.ndim == 3
    W, k = table.shape[-1], 0
    count = min(max(count, 0), len(free))
    for b in range(len(seq)):
        for dd in range(Dn if local else 1):
            t, h = (table[dd, b], (dd, b)) if local else (table[b], b)
            L = max(0, int(seq[b]))
            want = -(-(owned(L, d0 + dd, D, I) if local else L) // bs)
            if want > W:
                err, want = err | dcp.DEVERR_SEQ_TOO_LONG, W
            for col in range(max(0, int(held[h])), want):
                t[col] = free[count - 1 - k] if k < count else -1
                held[h] = col + 1 if k < count else max(0, int(held[h]))
                k += 1
    pos, slots = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    for b in range(len(seq)):
        L, n = int(seq[b]), int(qsl[b + 1] - qsl[b])
        for i in range(n):
            p, r = L - n + i, int(qsl[b]) + i
            if L <= 0 or p < 0 or r >= T:
                continue
            pos[r] = p
            d = (p // I) % D
            if d0 <= d < d0 + Dn:
                j = p // (D * I) * I + p % I if local else p
                if j // bs < W:
                    blk = int((table[d - d0, b] if local else table[b])[j // bs])
                    slots[r] = blk * bs + j % bs if blk >= 0 else -1
    if k > count:
        err |= dcp.DEVERR_NO_BLOCKS
    return table, held, pos, slots, max(0, count - k), err


class Run:
    def __init__(self, B, W, bs, D=1, I=1, d0=0, Dn=None, local=False, blocks=300, seed=0):
        self.D, self.I, self.d0, self.Dn, self.bs, self.local = D, I, d0, D if Dn is None else Dn, bs, local
        rng = np.random.default_rng(seed)
        self.free_h, self.left = rng.permutation(blocks).astype(np.int32), blocks
        lead = (self.Dn, B) if local else (B,)
        self.table_h, self.held_h = np.full(lead + (W,), -1, np.int32), np.zeros(lead, np.int32)
        self.free = torch.from_numpy(self.free_h).cuda()
        self.count = torch.tensor([blocks], dtype=torch.int32, device="cuda")
        self.table, self.held = torch.from_numpy(self.table_h).cuda(), torch.from_numpy(self.held_h).cuda()
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step(self, seq, q, pad=0):
        """One step, checked against the definition; returns its slots and error."""
        seq, qsl = np.asarray(seq, np.int32), np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        T = int(qsl[-1]) + pad
        want = expected(self.table_h, self.held_h, seq, qsl, self.free_h, self.left, T, self.bs, self.D, self.I, self.d0,
                        self.Dn)
        self.err.zero_()
        pos, slots = dcp.cache_extend(self.table, torch.from_numpy(seq).cuda(), torch.from_numpy(qsl).cuda(), self.free,
                                      self.count, T, self.bs, D=self.D, interleave=self.I, shard_begin=self.d0,
                                      shard_count=self.Dn, held=self.held, dev_error=self.err)
        got = (self.table.cpu().numpy(), self.held.cpu().numpy(), pos.cpu().numpy(), slots.cpu().numpy())
        for g, w in zip(got, want):
            assert np.array_equal(g, w)
        assert (int(self.count), int(self.err)) == want[4:]
        self.table_h, self.held_h, self.left = want[0], want[1], want[4]
        in_use = self.table_h[np.arange(self.table_h.shape[-1]) < self.held_h[..., None]]
        assert len(set(in_use.tolist())) == len(in_use)  # no block twice, and none lost:
        assert set(in_use.tolist()) | set(self.free_h[:self.left].tolist()) >= set(self.all_blocks())
        return want[3], want[5]

    def all_blocks(self):
        return self.free_h.tolist()


def test_rejected_drafts_keep_their_blocks():
    """62 tokens and four draft rows reach into a second block; one draft is accepted a
    step, and the block stays the request's."""
    r = Run(1, 4, 64, blocks=20)
    r.step([62], [62])
    r.step([66], [4])
    assert r.left == 18
    block = int(r.table_h[0, 1])
    for seq in (67, 68, 69, 130):  # old = 63, 64, 65, 126
        r.step([seq], [4])
        assert int(r.table_h[0, 1]) == block
    assert r.left == 17


@pytest.mark.parametrize("D,I,d0,Dn,local", [(1, 1, 0, 1, False), (8, 1, 0, 8, True), (3, 5, 0, 3, True), (4, 3, 1, 2, True),
                                             (4, 3, 2, 1, False)])
@pytest.mark.parametrize("B", [1, 37, 700])
def test_verification_steps(D, I, d0, Dn, local, B):
    """Requests of any lengths verify 1 to 5 drafts a step and keep some of them."""
    rng = np.random.default_rng(B)
    r = Run(B, 60, 4, D, I, d0, Dn, local, blocks=60 * B * (Dn if local else 1) + 5)
    ctx = rng.integers(0, 60, B)
    q = np.maximum(ctx, 1)
    r.step(q, q, pad=3)
    ctx = q
    for _ in range(6):
        q = rng.integers(1, 6, B)
        r.step(ctx + q, q, pad=2)
        ctx = ctx + rng.integers(0, q + 1)  # accepted


def test_blocks_missing_after_the_list_ran_out_come_later():
    r = Run(2, 8, 16, blocks=5)
    slots, err = r.step([60, 40], [60, 40])  # 4 + 3 blocks of 5
    assert err == dcp.DEVERR_NO_BLOCKS and r.left == 0 and r.held_h.tolist() == [4, 1]
    # request 0 is finished: its blocks go back, its table starts again
    back = r.table_h[0, :4].copy()
    r.free_h[:4] = back
    r.free[:4] = torch.from_numpy(back).cuda()
    r.left = 4
    r.count.fill_(4)
    r.held_h[0] = 0
    r.held[0] = 0
    slots, err = r.step([0, 41], [0, 1])
    assert err == 0 and r.held_h.tolist() == [0, 3] and r.left == 2 and slots[0] >= 0


@pytest.mark.parametrize("T_pad", [0, 4000])
def test_bounds_strides_and_graphs(T_pad):
    """Counts past the width or below 0; a table narrower than its request; replayed."""
    r = Run(3, 4, 16, blocks=50)
    r.table_h[:] = np.arange(12).reshape(3, 4) + 100
    r.table.copy_(torch.from_numpy(r.table_h))
    r.held_h[:] = r.held[:] = torch.tensor([9, -3, 2], dtype=torch.int32)
    r.held.copy_(torch.from_numpy(r.held_h))
    r.all_blocks = lambda: []
    _, err = r.step([70, 20, 90], [3, 20, 30], pad=T_pad)
    assert err == dcp.DEVERR_SEQ_TOO_LONG
    seq, qsl = torch.tensor([40, 23, 64], dtype=torch.int32, device="cuda"), torch.tensor([0, 1, 4, 5], dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dcp.cache_extend(r.table, seq, qsl, r.free, r.count, 5 + T_pad, 16, held=r.held)
    for lens in ([40, 23, 64], [64, 40, 64], [64, 41, 64]):
        seq.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        want = expected(r.table_h, r.held_h, np.array(lens), np.array([0, 1, 4, 5]), r.free_h, r.left, 5 + T_pad, 16, 1, 1, 0, 1)
        assert np.array_equal(r.table.cpu().numpy(), want[0]) and np.array_equal(r.held.cpu().numpy(), want[1])
        assert int(r.count) == want[4]
        r.table_h, r.held_h, r.left = want[0], want[1], want[4]


def test_without_a_count_as_before():
    """No count: the columns past the old tokens, whatever they hold."""
    free, count = torch.arange(20, dtype=torch.int32, device="cuda"), torch.tensor([20], dtype=torch.int32, device="cuda")
    table = torch.full((1, 4), 99, dtype=torch.int32, device="cuda")
    seq, qsl = torch.tensor([67], dtype=torch.int32, device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
    dcp.cache_extend(table, seq, qsl, free, count, 4, 64)
    assert table.tolist() == [[99, 19, 99, 99]] and int(count) == 19
