"""Every tensor of the full-attention calls at an address that is 16 bytes off a multiple of 32: the
alignment the header asks for and no more.  Each result is compared, bit for bit, with that of
the allocator's own (256-byte aligned) buffers, and the bytes beside each buffer stay as they were."""
import pytest
import torch

from tests import dense_cases as dc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa(cuda_device):
    import block_sparse_long_branch_b200 as m
    m.load_library()
    return m


class Shifted:
    """Copies of tensors 16 bytes into buffers of their own, between guard bytes."""

    def __init__(self):
        self.guards = []

    def __call__(self, t):
        n = t.numel() * t.element_size()
        raw = torch.full((n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
        at = (16 - raw.data_ptr()) % 32
        self.guards += [raw[:at], raw[at + n:]]
        view = raw[at:at + n].view(t.dtype).view(t.shape)
        view.copy_(t)
        assert view.data_ptr() % 32 == 16
        return view

    def untouched(self):
        return all(bool((g == 0xA5).all()) for g in self.guards)


def scratch(msa, cfg, op, T, B):
    return torch.full((msa.msa_workspace_size(cfg, op, T, B),), 0xFF, dtype=torch.uint8,
                      device="cuda")


@pytest.mark.parametrize("H,G,d,lens", [
    (8, 2, 128, [100, 28]),          # a few units, written whole
    (4, 2, 64, [300, 1, 0, 77]),
    (1, 1, 128, [2600]),             # split along the keys and joined
    (2, 2, 64, [1900, 3, 700]),
    (8, 8, 64, [2600, 2100]),        # planned on the device
])
def test_packed_prefill(msa, H, G, d, lens):
    cu = dc.offsets(lens)
    T = cu[-1]
    cfg = msa.config(H, G, d, d)
    q, k, v = (dc.randn((T, n, d), 3 + i) for i, n in enumerate((H, G, G)))
    want = msa.msa_dense_prefill_varlen(cfg, q, k, v, cu)
    at16 = Shifted()
    out = at16(torch.zeros_like(q))
    ws = at16(scratch(msa, cfg, msa.OP_DENSE_PREFILL, T, len(lens)))
    msa.msa_dense_prefill_varlen(cfg, at16(q), at16(k), at16(v), cu, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    assert torch.equal(out, want) and at16.untouched()


@pytest.mark.parametrize("H,G,d,new,ctx", [
    (8, 2, 128, [5, 40], [30, 200]),                   # units written whole
    (8, 1, 128, [3, 8], [5000, 2111]),                 # parts, joined
    (16, 2, 64, [700, 560, 3], [4200, 3600, 9000]),    # even shares, joined
    (8, 2, 64, [70] + [2] * 39, [9000] + [50] * 39),   # planned on the device, one unit split
])
def test_paged_prefill(msa, H, G, d, new, ctx):
    lens = [c + n for c, n in zip(ctx, new)]
    k, v, table, _ = dc.pool(lens, 32, G, d, 6)
    cu = torch.tensor(dc.offsets(new)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    T = sum(new)
    cfg = msa.config(H, G, d, d)
    q = dc.randn((T, H, d), 4)
    want = msa.msa_dense_prefill_paged(cfg, q, msa.paged_kv(k, v, table), cu, sl)
    at16 = Shifted()
    out = at16(torch.zeros_like(q))
    ws = at16(scratch(msa, cfg, msa.OP_DENSE_PREFILL_PAGED, T, len(new)))
    msa.msa_dense_prefill_paged(cfg, at16(q), msa.paged_kv(at16(k), at16(v), at16(table)),
                                at16(cu), at16(sl), out=out, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    assert torch.equal(out, want) and at16.untouched()


@pytest.mark.parametrize("H,G,d,lens", [(8, 2, 128, [300, 1, 0]), (32, 1, 64, [6000]),
                                        (64, 8, 128, [9000, 17, 12000])])
def test_paged_decode(msa, H, G, d, lens):
    k, v, table, _ = dc.pool(lens, 16, G, d, 8)
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    B = len(lens)
    cfg = msa.config(H, G, d, d)
    q = dc.randn((B, H, d), 5)
    want = msa.msa_dense_decode_paged(cfg, q, msa.paged_kv(k, v, table), sl)
    at16 = Shifted()
    out = at16(torch.zeros_like(q))
    ws = at16(scratch(msa, cfg, msa.OP_DENSE_DECODE, B, B))
    msa.msa_dense_decode_paged(cfg, at16(q), msa.paged_kv(at16(k), at16(v), at16(table)), at16(sl),
                               out=out, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    assert torch.equal(out, want) and at16.untouched()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,G,d", [(8, 2, 128), (3, 1, 64)])
def test_append(msa, H, G, d, interleaved):
    new, ctx, page = [5, 33], [20, 0], 16
    lens = [c + n for c, n in zip(ctx, new)]
    cfg = msa.config(H, G, d, d)
    T = sum(new)
    q, k, v = (dc.randn((T, n, d), 3 + i) for i, n in enumerate((H, G, G)))
    w = (10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)).float().cuda()
    kc, vc, table, _ = dc.pool(lens, page, G, d, 2, fill=3.0)
    cu = torch.tensor(dc.offsets(new)).cuda()
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    at16 = Shifted()
    kc2, vc2, qo = at16(kc), at16(vc), at16(torch.zeros_like(q))
    ws = at16(scratch(msa, cfg, msa.OP_ROPE_APPEND, T, 2))
    want = msa.msa_rope_append_paged(cfg, q, k, v, w, msa.paged_kv(kc, vc, table), cu, sl,
                                     interleaved=interleaved)
    msa.msa_rope_append_paged(cfg, at16(q), at16(k), at16(v), at16(w),
                              msa.paged_kv(kc2, vc2, at16(table)), at16(cu), at16(sl),
                              interleaved=interleaved, q_out=qo, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    assert torch.equal(qo, want) and torch.equal(kc2, kc) and torch.equal(vc2, vc)
    assert at16.untouched()
