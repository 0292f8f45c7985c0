"""The full-attention operators as a serving loop uses them: append and prefill in chunks, then
decode steps, direct and from CUDA graphs, on side streams."""
import numpy as np
import pytest
import torch

from oracle import dense
from tests import dense_cases as dc
from tests.dense_cases import check_rotated

pytestmark = pytest.mark.gpu

H, G, D, PAGE, COLS = 8, 2, 128, 16, 24
BASE = 10000.0


@pytest.fixture(scope="module")
def msa(cuda_device):
    import block_sparse_long_branch_b200 as m
    m.load_library()
    return m


class Server:
    """A cache for three sequences whose pages are handed out in a random order."""

    def __init__(self, msa):
        self.msa = msa
        self.cfg = msa.config(H, G, D, D)
        self.B = 3
        self.tnp = np.random.default_rng(2).permutation(self.B * COLS).astype(np.int32)
        self.tnp = self.tnp.reshape(self.B, COLS)
        self.table = torch.from_numpy(self.tnp).cuda()
        self.kc = torch.full((self.B * COLS, PAGE, G, D), float("nan"), dtype=torch.bfloat16,
                             device="cuda")
        self.vc = self.kc.clone()
        self.kv = msa.paged_kv(self.kc, self.vc, self.table)
        self.w = (BASE ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
        self.lens = [0] * self.B

    def check_append(self, q, k, v, qr, new):
        """The rotated queries and the rows the cache now holds; advances the lengths."""
        cu = dc.offsets(new)
        for b, n in enumerate(new):
            a, e = cu[b], cu[b + 1]
            pos = np.arange(self.lens[b], self.lens[b] + n)
            pg, row = torch.from_numpy(self.tnp[b, pos // PAGE].astype(np.int64)), pos % PAGE
            check_rotated(qr[a:e], q[a:e], pos, self.w, False)
            check_rotated(self.kc[pg, row], k[a:e], pos, self.w, False)
            assert torch.equal(self.vc[pg, row], v[a:e])
            self.lens[b] += n

    def check_attention(self, out, qr, new, p_round):
        """Against fp64 attention of the rotated queries over the cache's rows."""
        cu = dc.offsets(new)
        ref, mag = dense.prefill_paged(qr[:cu[-1]], self.kc, self.vc, self.tnp, cu, self.lens,
                                       self.cfg.softmax_scale)
        dc.check_attention(out, ref, mag, dense.as_f64(qr[:cu[-1]]), dense.as_f64(self.kc),
                           self.cfg.softmax_scale, max(self.lens), p_round)


def tokens(new, seed):
    T = sum(new)
    qkv = dc.randn((T, (H + 2 * G) * D), seed)
    return (qkv[:, :H * D].view(T, H, D), qkv[:, H * D:(H + G) * D].view(T, G, D),
            qkv[:, (H + G) * D:].view(T, G, D))


def test_chunks_then_decode_steps(msa):
    s = Server(msa)
    for step, new in enumerate(([40, 1, 130], [17, 64, 0], [1, 1, 1], [1, 1, 1])):
        q, k, v = tokens(new, 30 + step)
        cu = torch.tensor(dc.offsets(new)).cuda()
        sl = torch.tensor([a + n for a, n in zip(s.lens, new)], dtype=torch.int32).cuda()
        qr = msa.msa_rope_append_paged(s.cfg, q, k, v, s.w, s.kv, cu, sl)
        out = msa.msa_dense_prefill_paged(s.cfg, qr, s.kv, cu, sl)
        s.check_append(q, k, v, qr, new)
        s.check_attention(out, qr, new, dc.HALF_BF16)
        if min(new) == max(new) == 1:
            s.check_attention(msa.msa_dense_decode_paged(s.cfg, qr, s.kv, sl), qr, new, 2.0 ** -16)


def test_two_graphs_share_a_workspace_and_follow_the_lengths(msa):
    """A chunk graph and a decode graph, captured once with one workspace, replayed in turn with
    new inputs and lengths written into the captured buffers."""
    s = Server(msa)
    size = max(msa.msa_workspace_size(s.cfg, msa.OP_DENSE_PREFILL_PAGED, 24, 3),
               msa.msa_workspace_size(s.cfg, msa.OP_DENSE_DECODE, 3, 3))
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device="cuda")
    bufs = {}
    for name, T in (("chunk", 24), ("step", 3)):
        bufs[name] = dict(qkv=torch.zeros((T, (H + 2 * G) * D), dtype=torch.bfloat16, device="cuda"),
                          cu=torch.tensor([0, 1, 2, 3]).cuda(),
                          sl=torch.ones(3, dtype=torch.int32).cuda(),
                          qr=torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda"),
                          out=torch.empty((T, H, D), dtype=torch.bfloat16, device="cuda"), T=T)

    def launch(name):
        x = bufs[name]
        T = x["T"]
        q = x["qkv"][:, :H * D].view(T, H, D)
        k = x["qkv"][:, H * D:(H + G) * D].view(T, G, D)
        v = x["qkv"][:, (H + G) * D:].view(T, G, D)
        msa.msa_rope_append_paged(s.cfg, q, k, v, s.w, s.kv, x["cu"], x["sl"], q_out=x["qr"],
                                  workspace=ws)
        if name == "chunk":
            msa.msa_dense_prefill_paged(s.cfg, x["qr"], s.kv, x["cu"], x["sl"], out=x["out"],
                                        workspace=ws)
        else:
            msa.msa_dense_decode_paged(s.cfg, x["qr"], s.kv, x["sl"], out=x["out"], workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        launch("chunk"), launch("step")
    torch.cuda.current_stream().wait_stream(side)
    graphs = {}
    for name in bufs:
        graphs[name] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graphs[name]):
            launch(name)
    s.kc.fill_(float("nan")), s.vc.fill_(float("nan"))
    for i, (name, new) in enumerate((("chunk", [10, 3, 8]), ("step", [1, 1, 1]),
                                     ("chunk", [1, 20, 3]), ("step", [1, 1, 1]),
                                     ("step", [1, 1, 1]))):
        x = bufs[name]
        q, k, v = tokens(new, 90 + i)
        T = sum(new)
        x["qkv"][:T] = torch.cat([t.reshape(T, -1) for t in (q, k, v)], 1)
        x["cu"].copy_(torch.tensor(dc.offsets(new)))
        x["sl"].copy_(torch.tensor([a + n for a, n in zip(s.lens, new)], dtype=torch.int32))
        x["out"].fill_(2.0)
        graphs[name].replay()
        torch.cuda.synchronize()
        assert msa.msa_get_device_error(ws) == 0
        s.check_append(q, k, v, x["qr"][:T], new)
        s.check_attention(x["out"][:T], x["qr"], new,
                          dc.HALF_BF16 if name == "chunk" else 2.0 ** -16)
        assert (x["out"][T:] == 2.0).all()
    graphs.clear()


def test_side_stream_with_binding_allocations(msa):
    """Calls on a stream of their own, workspaces and outputs left to the binding, several in
    flight: every result is the one of the current stream."""
    lens, new = [300, 77], [20, 5]
    k, v, table, _ = dc.pool(lens, PAGE, G, D, 12)
    kv = msa.paged_kv(k, v, table)
    cfg = msa.config(H, G, D, D)
    q = dc.randn((25, H, D), 4)
    qd = dc.randn((2, H, D), 6)
    cu, sl = torch.tensor([0, 20, 25]).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    pk, pv = dc.randn((25, G, D), 7), dc.randn((25, G, D), 8)
    want = (msa.msa_dense_prefill_paged(cfg, q, kv, cu, sl), msa.msa_dense_decode_paged(cfg, qd, kv, sl),
            msa.msa_dense_prefill_varlen(cfg, q, pk, pv, [0, 20, 25]))
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        a = msa.msa_dense_prefill_paged(cfg, q, kv, cu, sl, stream=s1)
        b = msa.msa_dense_decode_paged(cfg, qd, kv, sl, stream=s2)
        c = msa.msa_dense_prefill_varlen(cfg, q, pk, pv, [0, 20, 25], stream=s1)
        torch.cuda.synchronize()
        assert torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(c, want[2])
