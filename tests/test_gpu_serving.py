"""The serving operators run together, as a decode loop uses them: on the
default stream, on another stream, captured into a graph and replayed while
lengths grow, and two graphs side by side; against the oracle run the same way."""
import numpy as np
import pytest
import torch

from exact_attention_attn_gb300 import (attn_fwd_kv4, attn_fwd_status, attn_kv4_append, attn_kv4_cache, attn_kv4_read,
                                        attn_pages_assign, attn_pages_release, attn_rope, attn_rope_axes,
                                        attn_rope_table)
from exact_attention_attn_gb300.workloads import to_f64
from oracle import serving as S

from test_gpu_kv4 import _check_attention

pytestmark = pytest.mark.gpu

Hq, H, D, P = 8, 2, 128, 16
SECTIONS = (24, 20, 20)


def _dev(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


class Server:
    """Requests in a paged cache, stepped on the device; and what the oracle holds of the same state."""

    def __init__(self, B, width, pages, max_tokens, seed):
        self.B, self.T = B, max_tokens
        self.cache = attn_kv4_cache(pages, H, D, P)
        self.table, self.lens = _dev(np.full((B, width), -1)), _dev(np.zeros(B))
        self.free, self.count = _dev(np.random.default_rng(seed).permutation(pages)), _dev([pages])
        self.new = _dev(np.zeros(B))
        self.rope = attn_rope_table(D, SECTIONS)
        z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.q, self.k, self.v = z(max_tokens, Hq, D), z(max_tokens, H, D), z(max_tokens, H, D)
        self.out = {"lens": self.lens, "free_count": self.count}
        self.o, self.lse = z(max_tokens, Hq, D), torch.zeros((max_tokens, Hq), device="cuda")
        self.o_table, self.o_lens = np.full((B, width), -1), np.zeros(B, dtype=np.int64)
        self.o_free, self.o_count = self.free.cpu().numpy(), pages
        self.seed = seed

    def step(self, stream=None):
        s = attn_pages_assign(self.table, self.lens, self.new, self.free, self.count, P, self.T, out=self.out, stream=stream)
        self.out = s  # the same buffers every step
        pos = s["positions"][None, None].expand(3, 1, self.T)
        q4, k4 = self.q.transpose(0, 1)[None], self.k.transpose(0, 1)[None]
        attn_rope(q4, k4, pos, self.rope, out_q=q4, out_k=k4, stream=stream)
        attn_kv4_append(self.k, self.v, s["slots"], self.cache, P, stream=stream)
        attn_fwd_kv4(self.q, s["cu"], s["lens"], self.table, self.cache, P, out=self.o, lse=self.lse, stream=stream)

    def load(self, new):
        """The step's inputs; what the oracle expects of its state."""
        self.seed += 1
        g = torch.Generator().manual_seed(self.seed)
        for t in (self.q, self.k, self.v):
            t.copy_(torch.randn(t.shape, generator=g).to(torch.bfloat16))
        self.new.copy_(_dev(new))
        self.q0, self.k0 = self.q.clone(), self.k.clone()
        self.o.fill_(float("nan"))
        want = S.pages_assign(self.o_table, self.o_lens, np.asarray(new), self.o_free, self.o_count, P, self.T)
        assert want["info"][0] == 0
        self.o_table, self.o_lens, self.o_count = want["table"], want["lens"], want["free_count"]
        self.want = want

    def check(self):
        torch.cuda.synchronize()
        assert attn_fwd_status() == 0
        w, n = self.want, self.want["info"][1]
        for name in ("cu", "slots", "positions", "lens"):
            assert np.array_equal(self.out[name].cpu().numpy(), w[name]), name
        assert np.array_equal(self.table.cpu().numpy(), self.o_table) and self.count.item() == self.o_count
        inv, axis = [10000.0 ** (-2.0 * i / D) for i in range(D // 2)], attn_rope_axes(SECTIONS)
        pos = np.broadcast_to(w["positions"], (3, 1, self.T))
        for x0, x in ((self.q0, self.q), (self.k0, self.k)):
            want = S.rope(to_f64(x0).transpose(1, 0, 2)[None], pos, inv, axis)[0].transpose(1, 0, 2)
            assert np.abs(to_f64(x) - want).max() <= 2.0 ** -8 * np.abs(want).max() + 2.0 ** -17
        # the codes of this step's tokens, from the rotated k
        c, s, m, q = S.kv4_quantise(to_f64(self.k)[:n])
        gc, gs, gm = S.kv4_unpack(self.cache.cpu().numpy(), D, P)[0]
        at = w["slots"][:n]
        assert np.array_equal(gs[at // P, :, at % P], s) and np.array_equal(gm[at // P, :, at % P], m)
        differ = gc[at // P, :, at % P] != c
        assert (np.abs(q - np.floor(q) - 0.5)[differ] < 2.0 ** -19).all()
        _check_attention(self.o, self.lse, self.q, w["cu"], w["lens"], self.o_table, self.cache, D, P, D ** -0.5, True)
        assert torch.isnan(self.o[n:]).all()  # rows of the padding

    def release(self, keep):
        attn_pages_release(self.table, self.lens, _dev(keep), self.free, self.count, P,
                           out={"lens": self.lens, "free_count": self.count})
        back = S.pages_release(self.o_table, self.o_lens, keep, self.o_free, self.o_count, P)
        assert back["info"][0] == 0
        self.o_table, self.o_lens, self.o_free, self.o_count = back["table"], back["lens"], back["free"], back["free_count"]
        assert np.array_equal(self.free.cpu().numpy(), self.o_free) and np.array_equal(self.lens.cpu().numpy(), self.o_lens)


STEPS = [[60, 1, 0, 33], [1, 1, 1, 1], [1, 1, 20, 1], [4, 1, 1, 0], [0, 0, 0, 0]]


def test_decode_loop():
    s = Server(4, 12, 40, 100, seed=1)
    for i, new in enumerate(STEPS):
        s.load(new)
        s.step()
        s.check()
        if i == 2:  # a request ends, another takes back drafted tokens
            s.release([-1, 0, 7, -1])


def test_decode_loop_on_another_stream():
    s = Server(4, 12, 40, 100, seed=2)
    side = torch.cuda.Stream()
    for new in STEPS[:3]:
        s.load(new)
        side.wait_stream(torch.cuda.current_stream())
        s.step(stream=side)
        torch.cuda.current_stream().wait_stream(side)
        s.check()


def _capture(s):
    s.load([1, 1, 1, 1])
    s.step()
    s.check()
    g = torch.cuda.CUDAGraph()
    s.new.zero_()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        s.step()
    return g


def test_graph_replays_while_lengths_grow():
    s = Server(4, 300, 400, 120, seed=3)
    g = _capture(s)
    for new in ([100, 0, 3, 1], [1, 1, 1, 1], [1, 0, 0, 110], [1, 2, 3, 4]):
        s.load(new)
        g.replay()
        s.check()


def test_two_graphs_side_by_side():
    # two graphs replayed at once on two streams: each has its own workspace
    a, b = Server(4, 300, 400, 120, seed=4), Server(4, 300, 400, 120, seed=50)
    ga, gb = _capture(a), _capture(b)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for new in ([100, 0, 3, 1], [7, 90, 1, 1], [1, 1, 1, 1]):
        a.load(new)
        b.load(new[::-1])
        torch.cuda.synchronize()
        for g, st in ((ga, sa), (gb, sb)):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        a.check()
        b.check()


def test_steps_back_to_back_without_waiting():
    # many steps enqueued at once: the second kernel of one call overlaps the first's end, not the next call's reads
    s = Server(4, 100, 300, 8, seed=6)
    s.load([2, 1, 3, 1])
    s.step()
    s.check()
    outs, n = [], 30
    q = torch.randn((n, 8, Hq, D), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    for i in range(n):
        o, lse = attn_fwd_kv4(q[i], s.out["cu"], s.lens, s.table, s.cache, P)
        outs.append(o)
    torch.cuda.synchronize()
    for i in range(n):
        o, _ = attn_fwd_kv4(q[i], s.out["cu"], s.lens, s.table, s.cache, P)
        torch.cuda.synchronize()
        assert torch.equal(o[:7], outs[i][:7]), i


def test_two_streams_at_once():
    # the same operators on two streams without waiting for each other: their workspaces are their own
    a, b = Server(4, 100, 300, 60, seed=70), Server(4, 100, 300, 60, seed=90)
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for new in ([40, 3, 5, 9], [1, 1, 30, 1], [1, 1, 1, 1]):
        a.load(new)
        b.load(new[::-1])
        torch.cuda.synchronize()
        a.step(stream=sa)
        b.step(stream=sb)
        torch.cuda.synchronize()
        a.check()
        b.check()


def test_two_threads_at_once():
    import threading
    servers = [Server(4, 100, 300, 60, seed=110), Server(4, 100, 300, 60, seed=130)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in servers:
        s.load([40, 3, 5, 9])
    torch.cuda.synchronize()
    failed, ready = [], threading.Barrier(2)

    def run(s, stream):
        try:
            with torch.cuda.stream(stream):
                ready.wait(30)
                s.step()
                o, lse = s.o.clone(), s.lse.clone()
                n = s.want["info"][1]
                for _ in range(30):  # the same attention again, with outputs of its own
                    a, b = attn_fwd_kv4(s.q, s.out["cu"], s.lens, s.table, s.cache, P)
                    if not (torch.equal(a[:n], o[:n]) and torch.equal(b[:n], lse[:n])):
                        failed.append("differs")
        except Exception as e:  # noqa: BLE001
            failed.append(repr(e))

    threads = [threading.Thread(target=run, args=a) for a in zip(servers, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for s in servers:
        s.check()


@pytest.mark.parametrize("handle", [False, True])
def test_outputs_for_another_stream_take_no_block_in_use(handle):
    # a block whose last reader still waits on the current stream is not given to a call on another stream
    s = Server(4, 100, 300, 60, seed=37)
    s.load([40, 3, 5, 9])
    s.step()
    s.check()
    q4, slots, pos = s.q.transpose(0, 1)[None], s.out["slots"], s.out["positions"][None, None].expand(3, 1, s.T)
    table, side = s.table.clone(), torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    calls = {
        s.q.numel() * 2: lambda: attn_fwd_kv4(s.q, s.out["cu"], s.lens, s.table, s.cache, P, stream=stream),
        s.q.numel() * 2 + 1: lambda: attn_rope(q4, None, pos, s.rope, stream=stream),
        s.k.numel() * 2: lambda: attn_kv4_read(slots, s.cache, P, stream=stream),
        s.T * 4: lambda: attn_pages_assign(table, s.lens, s.new, s.free, s.count, P, s.T, stream=stream)}
    for size, call in calls.items():
        used = [torch.full((size,), 7, dtype=torch.uint8, device="cuda") for _ in range(8)]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)  # some 20 ms
        kept = [u.clone() for u in used]
        del used
        out = call()
        torch.cuda.synchronize()
        assert all((k == 7).all() for k in kept), size
        del out


def test_outputs_are_kept_for_the_other_stream():
    # outputs that the call allocates for a call on another stream are not handed out again before that stream is done
    s = Server(4, 100, 300, 60, seed=31)
    s.load([40, 3, 5, 9])
    s.step()
    s.check()
    want, _ = attn_fwd_kv4(s.q, s.out["cu"], s.lens, s.table, s.cache, P)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = []
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        o, lse = attn_fwd_kv4(s.q, s.out["cu"], s.lens, s.table, s.cache, P, stream=side)
        with torch.cuda.stream(side):
            got.append(o[:57].clone())
        del o, lse
        torch.full_like(s.q, 7.0)  # would land in the freed block
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[:57]) for g in got)
