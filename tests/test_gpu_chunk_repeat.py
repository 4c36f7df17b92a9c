"""The same call many times, next to other work on the GPU: the same bits.  (The
projection's pairs of CTAs hand each other weights, latents and accumulators;
a hand-over too early would show as another CTA's bits now and then.)"""
import pytest
import torch

from tests import chunk_reference as ref
import mla_decode_context_gb300 as dcp

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_many_calls_next_to_copies(fp8):
    st = ref.make(seq=[5000, 900, 300], q=[300, 200, 300], H=48, bs=64, fp8=fp8, seed=41)
    packed = dcp.pack_kv_b(st["w"])

    def call():
        return dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], packed, scale=st["scale"],
                                   total_len=st["total"], kv_scale=st["kv_scale"])
    out, lse = call()
    few = dict(st, H=2, q=st["q"][:, 46:].contiguous(), w=st["w"][46 * 256:].contiguous())
    ref.check(out[:, 46:].contiguous(), lse[:, 46:].contiguous(), ref.reference(few))
    side = torch.cuda.Stream()
    a = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    b = torch.empty_like(a)
    torch.cuda.synchronize()
    for i in range(60):
        if i % 3:
            with torch.cuda.stream(side):  # takes memory bandwidth, and SMs, from some of the calls
                b[:(i + 1) << 22].copy_(a[:(i + 1) << 22])
        o, l = call()
        assert torch.equal(o, out) and torch.equal(l, lse), i
    torch.cuda.synchronize()


def test_packed_weights_of_several_layers_in_one_graph():
    """Each call's copies read its own weight."""
    st = ref.make(seq=[300, 77], q=[50, 77], H=3, seed=42)
    weights = [dcp.pack_kv_b(st["w"] * s) for s in (1.0, -1.0, 2.0)]

    def call(w):
        return dcp.chunk_attention(st["q"], st["cache"], st["table"], st["seq"], st["qsl"], w, scale=st["scale"],
                                   total_len=st["total"], out_dtype=torch.float32)
    want = [call(w) for w in weights]
    assert not torch.equal(want[0][0], want[1][0]) and not torch.equal(want[0][0], want[2][0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [call(w) for w in weights]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    for (o, l), (wo, wl) in zip(got, want):
        assert torch.equal(o, wo) and torch.equal(l, wl)


def test_calls_from_two_threads():
    """Threads of their own streams and workspaces; the second's first call is its first
    use of the GPU."""
    import threading
    st = [ref.make(seq=[2500, 77], q=[50, 77], H=3, seed=43 + i) for i in range(2)]
    packed = [dcp.pack_kv_b(s["w"]) for s in st]

    def call(i, **kw):
        s = st[i]
        return dcp.chunk_attention(s["q"], s["cache"], s["table"], s["seq"], s["qsl"], packed[i], scale=s["scale"],
                                   total_len=s["total"], **kw)
    want = [call(i) for i in range(2)]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            stream = torch.cuda.Stream()
            for _ in range(20):
                o, l = call(i, stream=stream)
                stream.synchronize()
                if not (torch.equal(o, want[i][0]) and torch.equal(l, want[i][1])):
                    failed.append(i)
        except Exception as e:  # (a thread's exception is not the test's)
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
