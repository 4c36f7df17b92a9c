"""GPU parity of the windowed and tree decodes with the 64-bit oracle, on both
kernels, in both table layouts and cache formats: windows shorter and longer
than the contexts, sinks, causal verification chains, trees of one to 256
rows with odd masks, padding, groups of rows that share a unit, splits; then
what neither may touch (blocks outside every window, latents behind a mask),
poisoned and repeated calls, graphs, and the refusals the device reports.

Tolerances: the attention ones of the other decodes (outputs 1e-2 absolute,
LSE 1e-3), plus half a bf16 step (2^-8 of the value) for bf16 outputs."""
import numpy as np
import pytest
import torch

import oracle
import workloads as wl
import mla_decode_context_gb300 as dcp
from tests import gpu_util as G

pytestmark = pytest.mark.gpu


@pytest.fixture(params=["tc", "simt"])
def kernel(request, monkeypatch):
    if request.param == "simt":
        monkeypatch.setenv("DCP_FORCE_SIMT", "1")
    else:
        monkeypatch.delenv("DCP_FORCE_SIMT", raising=False)
    return request.param


def random_trees(rng, inp, kind="tree"):
    """Bool [T, max_q_len]: each request's rows as a random tree (a row sees
    itself and its ancestors), or ``odd``: any bits at all, empty rows, bits
    past the request's rows set."""
    qsl = inp["query_start_loc"]
    n = max(1, inp["max_q_len"])
    vis = np.zeros((inp["T"], n), dtype=bool)
    for b in range(inp["B"]):
        r0, q = int(qsl[b]), int(qsl[b + 1] - qsl[b])
        for i in range(q):
            if kind == "odd":
                vis[r0 + i] = rng.random(n) < rng.choice((0.0, 0.1, 0.6, 1.0))
            else:
                vis[r0 + i, i] = True
                if i:
                    vis[r0 + i] |= vis[r0 + rng.integers(max(0, i - 4), i)]
    return vis


def run(inp, t, window=0, sinks=0, tree=None, out_dtype=torch.float32, **kw):
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    args = dict(D=inp["D"], interleave=inp["interleave"], scale=inp["scale"], window=window, num_sinks=sinks,
                max_seq_len=max(1, inp["max_seq_len"]), max_q_len=max(1, inp["max_q_len"]), dev_error=err,
                kv_scale=t.get("kv_scale"), out_dtype=out_dtype)
    args.update(kw)
    ins = (t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["query_start_loc"])
    if tree is None:
        O, lse = dcp.decode_partial_window(*ins, **args)
    else:
        O, lse = dcp.decode_partial_tree(*ins, dcp.pack_tree_mask(torch.from_numpy(tree)).cuda(), **args)
    torch.cuda.synchronize()
    return O, lse, int(err.item())


def check(inp, O, lse, ref, what):
    O_ref, lse_ref = ref
    got, gl = O.float().cpu().numpy(), lse.cpu().numpy()
    if O.dtype == torch.float32:
        G.check_partials(got, gl, O_ref, lse_ref, what)
        return
    empty = lse_ref == -np.inf
    assert np.array_equal(gl == -np.inf, empty), what
    assert (got[empty] == 0).all(), what
    live = ~empty
    assert np.abs(gl[live] - lse_ref[live]).max(initial=0) <= G.ATT_LSE_ABS, what
    assert (np.abs(got[live] - O_ref[live]) <= G.ATT_OUT_ABS + 2.0 ** -8 * np.abs(O_ref[live])).all(), what


def S(name, **kw):
    kw.setdefault("block_size", 16)
    return wl.DecodeSpec(name, **kw)


# (spec, window, sinks)
WINDOWS = [
    (S("w100_s4_h128_d8", seed=1, B=3, seq_lens=(1, 700, 2049), H=128, block_size=64, D=8, interleave=1), 100, 4),
    (S("w3_s1_q4_padding", seed=2, B=4, seq_lens=(0, 2, 903, 4), q_len=4, H=128, D=2, extra_rows=2), 3, 1),
    (S("w37_s5_ragged_h16_i3_local", seed=3, B=3, seq_lens=(250, 40, 7), q_len=(1, 3, 7), H=16, D=4, interleave=3,
       layout="local"), 37, 5),
    (S("w_past_context", seed=4, B=2, seq_lens=(65, 300), q_len=2, H=64, D=3), 1000, 0),
    (S("w1_self_only", seed=5, B=2, seq_lens=(65, 9), q_len=3, H=8, D=8), 1, 0),
    (S("w0_everything", seed=6, B=2, seq_lens=(65, 300), q_len=5, H=16, D=2, interleave=64), 0, 7),
    (S("sinks_past_context", seed=7, B=3, seq_lens=(5, 40, 200), q_len=6, H=33, D=2), 2, 60),
    (S("sinks_meet_window", seed=8, B=1, seq_lens=(100,), q_len=8, H=16, D=1), 90, 8),
    (S("one_split_block_size_1", seed=9, B=1, seq_lens=(9000,), H=128, block_size=1, D=2), 5000, 3),
    (S("h1_q20", seed=10, B=2, seq_lens=(500, 19), q_len=20, H=1, D=1), 40, 2),
    (S("h160", seed=11, B=2, seq_lens=(90, 300), q_len=2, H=160, D=2), 50, 2),
    (S("fp8_w200", seed=12, B=3, seq_lens=(33, 500, 0), q_len=(1, 4, 2), H=128, D=4, kv_dtype="fp8_e4m3"), 200, 4),
    (S("fp8_h16_local", seed=13, B=2, seq_lens=(700, 81), q_len=5, H=16, D=2, interleave=5, layout="local",
       kv_dtype="fp8_e4m3"), 64, 1),
    (S("h100_q2_w31", seed=14, B=2, seq_lens=(400, 64), q_len=2, H=100, D=1), 31, 0),
]

# (spec, window, sinks, kind)
TREES = [
    (S("n7_h128", seed=21, B=1, seq_lens=(900,), q_len=7, H=128, block_size=64, D=1), 0, 0, "tree"),
    (S("n16_h16_ragged", seed=22, B=3, seq_lens=(300, 16, 47), q_len=(16, 5, 1), H=16, D=2), 0, 0, "tree"),
    (S("n70_h16_two_words", seed=23, B=2, seq_lens=(200, 70), q_len=70, H=16, D=1), 0, 0, "tree"),
    (S("n70_odd_i3_local", seed=24, B=2, seq_lens=(133, 90), q_len=(70, 66), H=8, D=4, interleave=3, layout="local"),
     0, 0, "odd"),
    (S("n256_h4", seed=25, B=1, seq_lens=(600,), q_len=256, H=4, D=2), 0, 0, "tree"),
    (S("n9_window", seed=26, B=2, seq_lens=(500, 60), q_len=9, H=128, D=2), 33, 2, "tree"),
    (S("n30_window_shorter_than_tree", seed=27, B=2, seq_lens=(100, 30), q_len=30, H=16, D=2), 3, 1, "odd"),
    (S("n12_sinks_in_tree", seed=28, B=2, seq_lens=(14, 12), q_len=12, H=16, D=1), 2, 6, "odd"),
    (S("tree_longer_than_context", seed=29, B=3, seq_lens=(4, 1, 0), q_len=9, H=16, D=2, extra_rows=3), 0, 0, "odd"),
    (S("odd_masks_h128", seed=30, B=2, seq_lens=(150, 40), q_len=6, H=128, D=8), 0, 0, "odd"),
    (S("fp8_n16_window", seed=31, B=2, seq_lens=(400, 17), q_len=16, H=128, D=2, interleave=64,
       kv_dtype="fp8_e4m3"), 100, 4, "tree"),
    (S("fp8_n61_h40", seed=32, B=2, seq_lens=(300, 100), q_len=(61, 2), H=40, D=1, kv_dtype="fp8_e4m3"), 0, 0, "tree"),
    (S("h130", seed=33, B=1, seq_lens=(120,), q_len=9, H=130, D=2), 20, 1, "odd"),
    (S("split", seed=34, B=1, seq_lens=(6000,), q_len=4, H=128, block_size=64, D=1), 0, 0, "tree"),
    (S("split_h16_window", seed=35, B=1, seq_lens=(6000,), q_len=20, H=16, block_size=64, D=1), 3000, 5, "tree"),
    (S("one_row", seed=36, B=3, seq_lens=(1, 33, 64), q_len=1, H=16, D=1), 0, 0, "odd"),
]


@pytest.mark.parametrize("case", WINDOWS, ids=lambda c: c[0].name)
def test_window_matches_oracle(case, kernel):
    spec, W, n = case
    inp = wl.make_decode_inputs(spec)
    t = G.to_device(inp)
    ref = oracle.decode_partial_select(inp, W, n)
    for dt in (torch.float32, torch.bfloat16):
        O, lse, err = run(inp, t, W, n, out_dtype=dt)
        assert err == 0
        check(inp, O, lse, ref, "%s/%s" % (spec.name, kernel))


@pytest.mark.parametrize("case", TREES, ids=lambda c: c[0].name)
def test_tree_matches_oracle(case, kernel):
    spec, W, n, kind = case
    inp = wl.make_decode_inputs(spec)
    t = G.to_device(inp)
    vis = random_trees(np.random.default_rng(spec.seed), inp, kind)
    ref = oracle.decode_partial_select(inp, W, n, vis)
    for dt in (torch.float32, torch.bfloat16):
        O, lse, err = run(inp, t, W, n, vis, out_dtype=dt)
        assert err == 0
        check(inp, O, lse, ref, "%s/%s" % (spec.name, kernel))


def test_chain_tree_is_the_plain_decode(kernel):
    """A lower-triangular mask is the causal chain: the same partials as the
    decode without selection, within twice the attention tolerance."""
    inp = wl.make_decode_inputs(S("chain", seed=41, B=2, seq_lens=(300, 80), q_len=4, H=128, D=2))
    t = G.to_device(inp)
    O, lse, _ = G.run_decode(inp, t)
    vis = np.tile(np.tril(np.ones((4, 4), bool)), (2, 1))
    for kw in (dict(tree=vis), dict()):
        O2, lse2, err = run(inp, t, **kw)
        assert err == 0
        assert (O - O2).abs().max().item() <= 2 * G.ATT_OUT_ABS
        assert (lse - lse2).abs().max().item() <= 2 * G.ATT_LSE_ABS


def test_partials_combine_to_the_whole(kernel):
    inp = wl.make_decode_inputs(S("comb", seed=42, B=3, seq_lens=(300, 0, 5), q_len=5, H=16, D=4, extra_rows=2))
    t = G.to_device(inp)
    vis = random_trees(np.random.default_rng(42), inp)
    O, lse, err = run(inp, t, 50, 3, vis)
    assert err == 0
    out, out_lse = G.run_combine(O, lse, t)
    _, _, pad = oracle.row_lengths(inp["seq_lens"], inp["query_start_loc"], inp["T"])
    ref = oracle.lse_combine(*oracle.decode_partial_select(inp, 50, 3, vis), pad)
    G.check_combined(out.float().cpu().numpy(), out_lse.cpu().numpy(), *ref, pad, "combined")


def test_blocks_outside_every_window_are_never_read(kernel):
    """Their table entries are garbage and their latents NaN; nothing is
    flagged and nothing changes."""
    spec = S("evicted", seed=43, B=2, seq_lens=(500, 200), q_len=3, H=16, D=2)
    inp = wl.make_decode_inputs(spec)
    W, n = 40, 2
    ref = oracle.decode_partial_select(inp, W, n)
    table = inp["block_table"].copy()
    kv = inp["kv_cache"].copy()
    for b, L in ((0, 500), (1, 200)):
        first = (L - 2 - W) // 16  # the block of the earliest window's first token
        kv[table[b, 1:first]] = wl.BF16_NAN
        table[b, 1:first] = (1 << 30, -5)[b]
    t = G.to_device(dict(inp, kv_cache=kv, block_table=table))
    O, lse, err = run(inp, t, W, n)
    assert err == 0
    check(inp, O, lse, ref, "evicted")


@pytest.mark.parametrize("H", [128, 16])
def test_latents_behind_a_mask_may_be_anything(kernel, H):
    """A tree token (then a window's departed token) that holds NaN or
    infinities changes no row that does not see it, also where rows that do
    share the unit."""
    spec = S("nan_h%d" % H, seed=44, B=1, seq_lens=(100,), q_len=8, H=H, D=1)
    inp = wl.make_decode_inputs(spec)
    base = 92
    for bad, fill in ((3, 0x7FC0), (5, 0x7F80), (6, 0xFF80)):
        vis = random_trees(np.random.default_rng(H + bad), inp)
        vis[:, bad] = False
        vis[bad, bad] = True  # only the row itself sees it
        ref = oracle.decode_partial_select(inp, 0, 0, vis)
        kv = inp["kv_cache"].copy()
        p = base + bad
        kv[inp["block_table"][0, p // 16], p % 16, 7:300:5] = fill
        t = G.to_device(dict(inp, kv_cache=kv))
        O, lse, err = run(inp, t, tree=vis)
        assert err == 0
        keep = np.arange(8) != bad
        got, gl = O.cpu().numpy()[:, keep], lse.cpu().numpy()[:, keep]
        G.check_partials(got, gl, ref[0][:, keep], ref[1][:, keep], "bad token %d" % bad)
        if fill == 0x7FC0:  # and the row that sees a NaN does not hide it
            assert np.isnan(O.cpu().numpy()[:, bad]).all() and np.isnan(lse.cpu().numpy()[:, bad]).all()
    # a chain's window: token 60 is behind the last rows' windows only
    kv = inp["kv_cache"].copy()
    kv[inp["block_table"][0, 60 // 16], 60 % 16] = 0x7FC0
    t = G.to_device(dict(inp, kv_cache=kv))
    W = 35  # row i sees [93 + i - 35, 93 + i)
    O, lse, err = run(inp, t, W, 0)
    keep = np.array([93 + i - W > 60 for i in range(8)])
    assert keep.any() and not keep.all() and err == 0
    ref = oracle.decode_partial_select(inp, W, 0)
    G.check_partials(O.cpu().numpy()[:, keep], lse.cpu().numpy()[:, keep], ref[0][:, keep], ref[1][:, keep], "chain")


def test_scores_far_apart(kernel):
    """Scores hundreds of bits apart (scale 1: a standard deviation of 24
    nats) and their order reversed (scale -1).  |ds| <= 370 * 2^-21 (the sum
    of 576 products of N(0, 1) pairs, 370 in magnitude, in fp32 with a few
    roundings to spare), and a weight is rounded to bf16 (2^-8), so an output
    is off by at most (2 |ds| + 2^-8) max |v|; LSE by |ds| and its own
    rounding."""
    inp = wl.make_decode_inputs(S("far", seed=45, B=2, seq_lens=(700, 333), q_len=5, H=16, D=2))
    t = G.to_device(inp)
    vis = random_trees(np.random.default_rng(45), inp)
    vmax = np.abs(oracle.bf16_to_f64(inp["kv_cache"][~np.isnan(oracle.bf16_to_f64(inp["kv_cache"]))])).max()
    ds = 370 * 2.0 ** -21
    for scale in (1.0, -1.0, 0.0):
        inp["scale"] = scale
        O, lse, err = run(inp, t, tree=vis)
        O_ref, lse_ref = oracle.decode_partial_select(inp, tree=vis)
        assert err == 0
        live = lse_ref != -np.inf
        assert np.abs(lse.cpu().numpy()[live] - lse_ref[live]).max() <= ds + 2.0 ** -23 * np.abs(lse_ref[live]).max()
        assert np.abs(O.cpu().numpy()[live] - O_ref[live]).max() <= (2 * ds + 2.0 ** -8) * vmax


def test_one_token_dwarfs_the_rest(kernel):
    """A late tile's score is 2^600 times everything else's, and the tiles
    after it fall back: neither overflows what was summed before."""
    inp = wl.make_decode_inputs(S("spike", seed=46, B=1, seq_lens=(640,), q_len=2, H=16, D=1))
    q = np.zeros((2, 16, 576), np.float32)
    q[:, :, 575] = 1.0
    bits = wl.f32_to_bf16_bits(q)
    for at in (0, 31, 70, 100, 133, 400, 637):
        x = oracle.bf16_to_f64(inp["kv_cache"]).copy()
        rows = np.concatenate([inp["block_table"][0, :40].astype(int)])
        x[rows, :, 575] = 0.0
        x[inp["block_table"][0, at // 16], at % 16, 575] = 416.0
        kv = wl.f32_to_bf16_bits(np.nan_to_num(x).astype(np.float32))
        i2 = dict(inp, q=bits, kv_cache=kv, scale=1.0)
        t = G.to_device(i2)
        O, lse, err = run(i2, t)
        ref = oracle.decode_partial_select(i2)
        assert err == 0
        # the one token's weight is 1: its values, rounded as P is
        assert np.abs(lse.cpu().numpy() - ref[1]).max() <= 416 * 2.0 ** -23
        assert (np.abs(O.cpu().numpy() - ref[0]) <= 2.0 ** -8 * np.abs(ref[0]) + 1e-6).all(), at


def test_calls_repeat_bit_for_bit_and_need_no_clean_memory():
    inp = wl.make_decode_inputs(S("rep", seed=47, B=2, seq_lens=(3000, 900), q_len=9, H=16, D=1, block_size=64))
    t = G.to_device(inp)
    vis = random_trees(np.random.default_rng(47), inp)
    n = dcp.dcp_decode_select_workspace_size(2, 18, 16, 1, 3000, 9, 1000, 2)
    assert n > 0
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")  # NaN patterns
    first = run(inp, t, 1000, 2, vis, workspace=ws)
    for _ in range(10):
        ws.fill_(255)
        O, lse, err = run(inp, t, 1000, 2, vis, workspace=ws)
        assert torch.equal(O, first[0]) and torch.equal(lse, first[1]) and err == 0


def test_two_streams_and_a_graph():
    """Calls of their own workspaces overlap on two streams, and a captured
    pair replays on new inputs."""
    inps = [wl.make_decode_inputs(S("s%d" % k, seed=50 + k, B=2, seq_lens=(2000, 300), q_len=4, H=16, D=2,
                                    block_size=64)) for k in range(2)]
    ts = [G.to_device(i) for i in inps]
    vis = [random_trees(np.random.default_rng(k), i) for k, i in enumerate(inps)]
    masks = [dcp.pack_tree_mask(torch.from_numpy(v)).cuda() for v in vis]
    kw = dict(D=2, interleave=1, scale=inps[0]["scale"], window=600, num_sinks=3, max_seq_len=2000, max_q_len=4)

    def call(k):
        t = ts[k]
        return dcp.decode_partial_tree(t["q"], t["kv_cache"], t["block_table"], t["seq_lens"], t["query_start_loc"],
                                       masks[k], **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [None, None]
    for rep in range(5):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[k] = call(k)
    torch.cuda.synchronize()
    for k in range(2):
        check(inps[k], *outs[k], oracle.decode_partial_select(inps[k], 600, 3, vis[k]), "stream %d" % k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        res = [call(0), call(1)]
    ts[0]["q"].copy_(ts[1]["q"])
    masks[0].copy_(masks[1])
    g.replay()
    torch.cuda.synchronize()
    i2, v2 = dict(inps[0], q=inps[1]["q"]), vis[1]
    check(i2, *res[0], oracle.decode_partial_select(i2, 600, 3, v2), "replayed")
    assert torch.equal(res[1][0], outs[1][0])


def test_device_reports(kernel):
    inp = wl.make_decode_inputs(S("rep", seed=61, B=2, seq_lens=(300, 80), q_len=4, H=16, D=1))
    t = G.to_device(inp)
    # a sequence past the declared bound: clamped
    O, lse, err = run(inp, t, 50, 1, max_seq_len=200)
    assert err == dcp.DEVERR_SEQ_TOO_LONG
    cut = dict(inp, seq_lens=np.minimum(inp["seq_lens"], 200))
    check(inp, O, lse, oracle.decode_partial_select(cut, 50, 1), "clamped")
    # more rows than declared: the rest is padding
    O, lse, err = run(inp, t, 50, 1, max_q_len=3)
    assert err == dcp.DEVERR_BAD_ROWS
    ref = oracle.decode_partial_select(inp, 50, 1)
    for r in (3, 7):
        ref[1][:, r], ref[0][:, r] = -np.inf, np.nan
    check(inp, O, lse, ref, "rows")
    # a bad block id inside the window: its tokens are skipped
    table = inp["block_table"].copy()
    table[1, 80 // 16 - 1] = inp["num_blocks"]
    t2 = G.to_device(dict(inp, block_table=table))
    O, lse, err = run(inp, t2, 10, 0)
    assert err == dcp.DEVERR_BAD_BLOCK
    assert (lse.cpu().numpy()[:, 7] == -np.inf).all()  # row 7 sees [70, 80) only: block 4
    check_rows = oracle.decode_partial_select(inp, 10, 0)
    G.check_partials(O.cpu().numpy()[:, :4], lse.cpu().numpy()[:, :4], check_rows[0][:, :4], check_rows[1][:, :4], "")


def test_speculative_step_end_to_end():
    """One step as a server runs it, on an fp8 cache: write the drafted tree's
    latents, tree decode over a window, combine; then read the request back
    and check it against what was written."""
    spec = S("step", seed=70, B=2, seq_lens=(200, 77), H=16, D=2, kv_dtype="fp8_e4m3")
    inp = wl.make_decode_inputs(spec)
    t = G.to_device(inp)
    rng = np.random.default_rng(70)
    n = 6
    room = [int(16 * (-(-s // 16)) - s) for s in (200, 77)]
    assert min(room) < n  # the tree needs new blocks
    extra = inp["num_blocks"]
    table = np.concatenate([inp["block_table"], np.full((2, 2), -1, np.int32)], axis=1)
    for b, s in enumerate((200, 77)):
        table[b, -(-s // 16)] = extra + b
    codes = np.concatenate([inp["kv_cache"], np.full((2, 16, 576), wl.FP8_NAN)])
    scale = np.concatenate([inp["kv_scale"], np.ones((2, 16), np.float32)])
    new = wl.f32_to_bf16_bits(rng.standard_normal((2 * n, 576), dtype=np.float32))
    pos = np.array([[s + k for k in range(n)] for s in (200, 77)])
    slots = np.take_along_axis(table.astype(np.int64), pos // 16, 1) * 16 + pos % 16
    q = wl.f32_to_bf16_bits(rng.standard_normal((2 * n, 16, 576), dtype=np.float32))
    codes_ref, scale_ref = oracle.concat_cache_fp8(new[:, :512], new[:, 512:], slots.reshape(-1), codes, scale)
    seq = np.array([200 + n, 77 + n], np.int32)
    step = dict(inp, q=q, kv_cache=codes_ref, kv_scale=scale_ref, block_table=table, seq_lens=seq,
                query_start_loc=np.array([0, n, 2 * n], np.int32), T=2 * n, max_q_len=n, max_seq_len=int(seq.max()))
    vis = random_trees(rng, step)
    dev = G.to_device(dict(step, kv_cache=codes, kv_scale=scale))
    qd, nd = G.bf16_tensor(q), G.bf16_tensor(new)
    dev["q"] = dcp.decode_concat_cache(qd[:, :, :512], qd[:, :, 512:], nd[:, :512], nd[:, 512:],
                                       torch.from_numpy(slots.reshape(-1)).cuda(), dev["kv_cache"],
                                       kv_scale=dev["kv_scale"])
    O, lse, err = run(step, dev, 64, 4, vis)
    assert err == 0
    out, out_lse = G.run_combine(O, lse, dev)
    O_ref, lse_ref = oracle.decode_partial_select(step, 64, 4, vis)
    pad = np.zeros(2 * n, bool)
    G.check_combined(out.float().cpu().numpy(), out_lse.cpu().numpy(), *oracle.lse_combine(O_ref, lse_ref, pad), pad, "step")
    cu = torch.tensor([0, 206, 206 + 83], dtype=torch.int32, device="cuda")
    back = dcp.latent_cache_read(dev["kv_cache"], dev["block_table"], cu, 289, kv_scale=dev["kv_scale"],
                                 out_dtype=torch.float32)
    want = oracle.cache_read(oracle.kv_rows_f64(step), table, 16, (0, 0), (0, 206, 289))
    assert np.array_equal(back.double().cpu().numpy(), want)
