"""Block tables and slot maps built on the GPU, against a loop over requests,
shards, columns and rows.  Whole numbers: equal."""
import numpy as np
import pytest
import torch

import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu


def owned(L, d, D, I):
    return (L // (D * I)) * I + min(max(L % (D * I) - d * I, 0), I)


def expected(table, seq, qsl, free, count, T, bs, D, I, d0, Dn):
    """(table, positions, slots, left, error) by the definition."""
    table, err = table.copy(), 0
    local = table.ndim == 3
    W, k = table.shape[-1], 0
    count = min(max(count, 0), len(free))
    pos, slots = np.full(T, -1, np.int64), np.full(T, -1, np.int64)
    for b in range(len(seq)):
        L, n = max(0, int(seq[b])), max(0, int(qsl[b + 1] - qsl[b]))
        for dd in range(Dn if local else 1):
            have, want = ((owned(x, d0 + dd, D, I) if local else x) for x in (max(0, L - n), L))
            have, want = -(-have // bs), -(-want // bs)
            if want > W:
                err, want = err | dcp.DEVERR_SEQ_TOO_LONG, W
            for col in range(have, want):
                (table[dd, b] if local else table[b])[col] = free[count - 1 - k] if k < count else -1
                k += 1
    for b in range(len(seq)):
        L, n = int(seq[b]), int(qsl[b + 1] - qsl[b])
        for i in range(n):
            p, r = L - n + i, int(qsl[b]) + i
            if L <= 0 or p < 0 or r >= T:
                continue
            pos[r] = p
            d = (p // I) % D
            if not d0 <= d < d0 + Dn:
                continue
            j = p // (D * I) * I + p % I if local else p
            if j // bs < W:
                blk = int((table[d - d0, b] if local else table[b])[j // bs])
                if blk >= 0:
                    slots[r] = blk * bs + j % bs
    if k > count:
        err |= dcp.DEVERR_NO_BLOCKS
    return table, pos, slots, max(0, count - k), err


def inputs(rng, ctx, q, bs, D, I, d0, Dn, local, W, pad=0, block_hi=1 << 20):
    B = len(ctx)
    shape = (Dn, B, W) if local else (B, W)
    table = np.full(shape, -1, np.int32)
    for b in range(B):
        for dd in range(Dn if local else 1):
            n = -(-(owned(ctx[b], d0 + dd, D, I) if local else ctx[b]) // bs)
            (table[dd, b] if local else table[b])[:n] = rng.integers(0, block_hi, min(n, W))
    seq = np.asarray(ctx) + np.asarray(q)
    qsl = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    return table, seq.astype(np.int32), qsl, int(qsl[-1]) + pad


def run(table, seq, qsl, free, count, T, bs, D, I, d0, Dn, **kw):
    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in
           dict(table=table, seq=seq, qsl=qsl, free=free, count=np.array([count], np.int32)).items()}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pos, slots = dcp.cache_extend(dev["table"], dev["seq"], dev["qsl"], dev["free"], dev["count"], T, bs, D=D,
                                  interleave=I, shard_begin=d0, shard_count=Dn, dev_error=err, **kw)
    torch.cuda.synchronize()
    return dev["table"].cpu().numpy(), pos.cpu().numpy(), slots.cpu().numpy(), int(dev["count"]), int(err)


def check(*args):
    got, want = run(*args), expected(*args)
    for g, w in zip(got[:3], want[:3]):
        assert np.array_equal(g, w)
    assert got[3:] == want[3:]


CASES = {  # ctx, q, bs, D, I, d0, Dn, local, spare columns, spare free, pad
    "one_token": ([999], [1], 64, 1, 1, 0, 1, False, 0, 5, 0),
    "first_token": ([0], [1], 64, 1, 1, 0, 1, False, 0, 0, 3),
    "block_border": ([63, 64, 65, 127], [1, 1, 1, 2], 64, 1, 1, 0, 1, False, 1, 1, 0),
    "no_rows": ([5, 17], [0, 0], 16, 1, 1, 0, 1, False, 0, 2, 2),
    "ragged_blocks_of_one": ([0, 3, 9], [7, 1, 30], 1, 1, 1, 0, 1, False, 2, 4, 1),
    "local_8": ([0, 100, 5, 777], [300, 1, 64, 9], 16, 8, 1, 0, 8, True, 1, 9, 0),
    "local_odd_interleave": ([10, 0, 50], [33, 21, 4], 4, 3, 5, 0, 3, True, 0, 0, 2),
    "local_some_shards": ([10, 0, 50], [33, 21, 4], 4, 4, 3, 1, 2, True, 0, 1, 2),
    "global_some_shards": ([10, 0, 50], [33, 21, 4], 4, 4, 3, 2, 1, False, 0, 1, 2),
    "long_period": ([10, 0, 500], [33, 21, 4], 16, 32, 1 << 30, 0, 32, True, 0, 1, 0),
    "long_period_later_shards": ([10], [33], 16, 32, 1 << 30, 3, 2, True, 1, 1, 0),
    "prefill_two_launches": ([0, 4000, 64], [2049, 700, 1500], 64, 8, 64, 0, 8, True, 0, 3, 7),
    "one_table_of_many_blocks": ([7], [5000], 1, 1, 1, 0, 1, False, 0, 0, 0),
    "many_requests": (list(range(2500)), [1 + i % 3 for i in range(2500)], 16, 1, 1, 0, 1, False, 0, 11, 5),
    "many_tables": ([7 * i for i in range(700)], [1] * 700, 16, 4, 1, 0, 4, True, 2, 0, 0),
}


def build(name, rng):
    ctx, q, bs, D, I, d0, Dn, local, spare, left, pad = CASES[name]
    widest = max((owned(c + n, d, D, I) if local else c + n) for c, n in zip(ctx, q) for d in range(d0, d0 + Dn))
    W = max(1, -(-widest // bs)) + spare
    table, seq, qsl, T = inputs(rng, ctx, q, bs, D, I, d0, Dn, local, W, pad)
    need = sum(q) + len(ctx) * Dn + left
    return [table, seq, qsl, rng.permutation(need).astype(np.int32), need, T, bs, D, I, d0, Dn]


@pytest.mark.parametrize("name", sorted(CASES))
def test_tables_slots_and_positions(name):
    check(*build(name, np.random.default_rng(7)))


@pytest.mark.parametrize("count", [0, 1, 5, -3, 10**6])
def test_free_list_runs_out(count):
    args = build("local_8", np.random.default_rng(8))
    args[4] = count
    check(*args)


def test_table_too_narrow_keeps_what_fits():
    rng = np.random.default_rng(9)
    table, seq, qsl, T = inputs(rng, [20, 0], [40, 90], 16, 1, 1, 0, 1, False, 3)
    check(table, seq, qsl, rng.permutation(50).astype(np.int32), 50, T, 16, 1, 1, 0, 1)


def test_padding_requests_and_rows_before_position_0():
    rng = np.random.default_rng(10)
    table, seq, qsl, T = inputs(rng, [20, 0, 9, 5], [4, 6, 3, 2], 16, 1, 1, 0, 1, False, 3, pad=4)
    seq[2], seq[1] = 0, 2  # a request of no tokens, and one of fewer tokens than rows
    check(table, seq, qsl, rng.permutation(50).astype(np.int32), 50, T, 16, 1, 1, 0, 1)


def test_block_past_32_bits_of_slots():
    rng = np.random.default_rng(11)
    table, seq, qsl, T = inputs(rng, [100], [30], 1024, 1, 1, 0, 1, False, 1, block_hi=3)
    table[0, 0] = (1 << 31) - 1
    check(table, seq, qsl, np.arange(4, dtype=np.int32), 4, T, 1024, 1, 1, 0, 1)


def test_free_list_past_its_length_is_not_read():
    args = build("first_token", np.random.default_rng(12))
    args[4] = 1 << 30
    check(*args)


def test_strided_tables_streams_and_steps():
    """Two steps in a row on a side stream, the count in place, out of a wider
    table whose other columns stay."""
    rng = np.random.default_rng(13)
    B, W = 5, 6
    big = torch.full((B, 11), -7, dtype=torch.int32, device="cuda")
    table = big[:, 2:2 + W]
    table.fill_(-1)
    free = torch.from_numpy(rng.permutation(64).astype(np.int32)).cuda()
    count = torch.tensor([64], dtype=torch.int32, device="cuda")
    host, left = np.full((B, W), -1, np.int32), 64
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ctx = np.array([0, 0, 0, 0, 0])
    for q in ([5, 17, 0, 33, 1], [1, 1, 40, 2, 16]):
        seq, qsl = (ctx + q).astype(np.int32), np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        want = expected(host, seq, qsl, free.cpu().numpy(), left, int(qsl[-1]), 16, 1, 1, 0, 1)
        with torch.cuda.stream(side):
            s, l = torch.from_numpy(seq).cuda(), torch.from_numpy(qsl).cuda()
        pos, slots = dcp.cache_extend(table, s, l, free, count, int(qsl[-1]), 16, stream=side)
        side.synchronize()
        host, left = want[0], want[3]
        assert np.array_equal(table.cpu().numpy(), host) and int(count) == left
        assert np.array_equal(pos.cpu().numpy(), want[1]) and np.array_equal(slots.cpu().numpy(), want[2])
        ctx = ctx + q
    assert (big[:, :2] == -7).all() and (big[:, 2 + W:] == -7).all()


@pytest.mark.parametrize("T", [6, 4000])
def test_captured_and_replayed(T):
    """A graph of two calls that share one free list, replayed with new lengths."""
    free = torch.arange(1000, dtype=torch.int32, device="cuda")
    count = torch.tensor([1000], dtype=torch.int32, device="cuda")
    seq = torch.zeros(2, dtype=torch.int32, device="cuda")
    qsl = torch.zeros(3, dtype=torch.int32, device="cuda")
    tables = [torch.full((2, 300), -1, dtype=torch.int32, device="cuda") for _ in range(2)]

    def step():
        return [dcp.cache_extend(t, seq, qsl, free, count, T, 16) for t in tables]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for q, ctx in (([2, 4], [0, 0]), ([3, 3], [30, 47])):
        hs, hq = np.array(ctx, np.int32) + np.array(q, np.int32), np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        seq.copy_(torch.from_numpy(hs))
        qsl.copy_(torch.from_numpy(hq))
        left, before = int(count), [t.cpu().numpy() for t in tables]
        graph.replay()
        torch.cuda.synchronize()
        for t, b, (pos, slots) in zip(tables, before, outs):
            want = expected(b, hs, hq, free.cpu().numpy(), left, T, 16, 1, 1, 0, 1)
            left = want[3]
            assert np.array_equal(t.cpu().numpy(), want[0])
            assert np.array_equal(pos.cpu().numpy(), want[1]) and np.array_equal(slots.cpu().numpy(), want[2])
        assert int(count) == left


def test_no_requests():
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    left = torch.tensor([9], dtype=torch.int32, device="cuda")
    pos, slots = dcp.cache_extend(e.view(0, 1), e, zero, torch.arange(4, dtype=torch.int32, device="cuda"),
                                  torch.full_like(zero, 3), 5, 16, free_left=left)
    assert (pos == -1).all() and (slots == -1).all() and int(left) == 3
