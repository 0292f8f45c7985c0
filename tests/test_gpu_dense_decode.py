"""Full attention of one new token per sequence over a paged cache, against fp64."""
import numpy as np
import pytest
import torch

from oracle import dense
from tests import dense_cases as dc

pytestmark = pytest.mark.gpu

P_TWO_PARTS = 2.0 ** -16


@pytest.fixture(scope="module")
def msa(cuda_device):
    import block_sparse_long_branch_b200 as m
    m.load_library()
    return m


def run(msa, H, G, d, page, lens, seed=1, **pool_kw):
    k, v, table, tnp = dc.pool(lens, page, G, d, seed, **pool_kw)
    B = len(lens)
    q = dc.randn((B, H, d), seed * 10 + 7)
    cfg = msa.config(H, G, d, d)
    ws = torch.full((msa.msa_workspace_size(cfg, msa.OP_DENSE_DECODE, B, B),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    kv = msa.paged_kv(k, v, table)
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    out = torch.full((B, H, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    msa.msa_dense_decode_paged(cfg, q, kv, sl, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    ref, mag = dense.decode_paged(q, k, v, tnp, lens, cfg.softmax_scale)
    dc.check_attention(out, ref, mag, dense.as_f64(q), dense.as_f64(k), cfg.softmax_scale,
                       max(max(lens), 1), P_TWO_PARTS)
    again = msa.msa_dense_decode_paged(cfg, q, kv, sl, workspace=ws)
    assert torch.equal(out, again)  # the join's order does not depend on timing
    return out


@pytest.mark.parametrize("H,G,d", [(8, 1, 128), (64, 8, 128), (5, 5, 64), (10, 2, 128),
                                   (24, 2, 64), (16, 1, 128), (40, 2, 64), (128, 1, 128)])
@pytest.mark.parametrize("lens", [[1], [0, 17, 16, 15], [300, 1, 0, 1000, 128]])
def test_shapes(msa, H, G, d, lens):
    run(msa, H, G, d, 16, lens)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(msa, page):
    run(msa, 16, 2, 128, page, [257, 31, 900, 64], table_cols=70)
    run(msa, 4, 2, 64, page, [500, 255], side_by_side=True)


def test_all_sequences_empty(msa):
    out = run(msa, 4, 2, 64, 16, [0, 0, 0])
    assert (out == 0).all()


def test_many_sequences(msa):
    """More sequences than one scan of the lengths takes (256 at a time), empty ones between."""
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 60, size=700).tolist()
    lens[3], lens[255], lens[256], lens[511] = 900, 700, 0, 333
    run(msa, 4, 1, 64, 16, lens)


@pytest.mark.parametrize("H,G,d,lens", [
    (16, 8, 128, [9000, 1, 17, 12000, 0, 400, 16000, 33, 2]),  # all eight groups at a time
    (10, 2, 64, [30000, 5, 20001]),                            # two
    (32, 1, 64, [40000, 100]),                                 # two chunks of 16 heads
    (12, 4, 128, [8000, 31000, 3]),                            # four
    (3, 3, 128, [25000, 16, 7000]),                            # one
])
def test_long_lines(msa, H, G, d, lens):
    """Enough steps that several groups are read at a time and shares end inside sequences."""
    run(msa, H, G, d, 64, lens, side_by_side=True)


def test_one_long_sequence_of_one_group(msa):
    """6000 keys of a single item: every CTA holds a share."""
    run(msa, 8, 1, 64, 32, [6000])


def test_odd_values(msa):
    """A NaN key and an infinite value inside a sequence reach that sequence's outputs only."""
    H, G, d, page = 4, 2, 64, 16
    lens = [40, 33]
    k, v, table, tnp = dc.pool(lens, page, G, d, 9)
    v[int(tnp[0, 1]), 3, 1, 5] = float("inf")
    q = dc.randn((2, H, d), 3)
    cfg = msa.config(H, G, d, d)
    kv = msa.paged_kv(k, v, table)
    sl = torch.tensor(lens, dtype=torch.int32).cuda()
    out = msa.msa_dense_decode_paged(cfg, q, kv, sl).double().cpu().numpy()
    odd = ~np.isfinite(out)
    assert odd[0, 2:, 5].all() and odd.sum() == 2
    k[int(tnp[1, 0]), 2, 0, 0] = float("nan")
    out = msa.msa_dense_decode_paged(cfg, q, kv, sl).double().cpu().numpy()
    assert np.isnan(out[1, :2]).all() and np.isfinite(out[1, 2:]).all()
    assert np.isfinite(out[0, :2]).all()


@pytest.mark.parametrize("H,G,d", [(4, 2, 64), (8, 1, 128), (32, 2, 128)])
def test_infinite_values_stay_infinite(msa, H, G, d):
    """One infinity among the values a row sees makes the output that infinity, not NaN, at
    whatever key and weight; infinities of both signs make it NaN."""
    page, lens = 16, [40, 700, 9]
    k, v, table, tnp = dc.pool(lens, page, G, d, 21)
    def put(b, s, col, x):
        v[int(tnp[b, s // page]), s % page, G - 1, col] = x
    for col in range(8, 40):  # every key of sequence 0 and of sequence 2 in turn
        put(0, col, col, float("inf"))
        put(2, col % 9, col, float("-inf"))
    put(1, 0, 1, float("inf")), put(1, 699, 2, float("-inf")), put(1, 350, 3, float("inf"))
    put(1, 10, 4, float("inf")), put(1, 690, 4, float("-inf"))
    q = dc.randn((3, H, d), 5)
    cfg = msa.config(H, G, d, d)
    out = msa.msa_dense_decode_paged(cfg, q, msa.paged_kv(k, v, table),
                                     torch.tensor(lens, dtype=torch.int32).cuda())
    ref, mag = dense.decode_paged(q, k, v, tnp, lens, cfg.softmax_scale)
    assert np.isinf(ref).sum() == (2 * 32 + 3) * (H // G) and np.isnan(ref).sum() == H // G
    dc.check_attention(out, ref, mag, dense.as_f64(q), dense.as_f64(k), cfg.softmax_scale,
                       max(lens), P_TWO_PARTS)


def test_bad_entries_are_recorded(msa):
    H, G, d, page = 4, 2, 64, 16
    lens = [40, 33, 20]
    k, v, table, tnp = dc.pool(lens, page, G, d, 9)
    q = dc.randn((3, H, d), 3)
    cfg = msa.config(H, G, d, d)
    ws = torch.empty(msa.msa_workspace_size(cfg, msa.OP_DENSE_DECODE, 3, 3), dtype=torch.uint8,
                     device="cuda")
    ref, mag = dense.decode_paged(q, k, v, tnp, lens, cfg.softmax_scale)

    def call(ls, tb):
        return msa.msa_dense_decode_paged(cfg, q, msa.paged_kv(k, v, tb),
                                          torch.tensor(ls, dtype=torch.int32).cuda(), workspace=ws)

    def good(out, rows):
        dc.check_attention(out[rows], ref[rows], mag[rows], dense.as_f64(q), dense.as_f64(k),
                           cfg.softmax_scale, 40, P_TWO_PARTS)
    for bad in (-5, k.shape[0], 2 ** 31 - 1):
        tb = table.clone()
        tb[1, 0] = bad
        out = call(lens, tb)
        assert msa.msa_get_device_error(ws) == 0x201
        good(out, [0, 2])
    for bad in (-1, table.shape[1] * page + 1, 2 ** 31 - 1):
        out = call([40, bad, 20], table)
        assert msa.msa_get_device_error(ws) == 0x201
        good(out, [0, 2])
        assert (out[1] == 0).all()
    good(call(lens, table), [0, 1, 2])
    assert msa.msa_get_device_error(ws) == 0


def test_offsets_past_32_bits(msa):
    """Pages more than 2^32 elements apart (one page at the end of a 9 GB buffer)."""
    H, G, d, page = 8, 2, 128, 64
    stride = 1 << 26
    pages = 66
    big = torch.empty(pages * stride, dtype=torch.bfloat16, device="cuda")
    k = big.as_strided((pages, page, G, d), (stride, G * d, d, 1))
    v = big.as_strided((pages, page, G, d), (stride, G * d, d, 1), 1 << 25)
    used = [65, 3, 64]
    L = 150
    for i, p in enumerate(used):
        k[p] = dc.randn((page, G, d), 100 + i)
        v[p] = dc.randn((page, G, d), 200 + i)
    table = np.array([used], dtype=np.int32)
    q = dc.randn((1, H, d), 3)
    cfg = msa.config(H, G, d, d)
    out = msa.msa_dense_decode_paged(cfg, q, msa.paged_kv(k, v, torch.from_numpy(table).cuda()),
                                     torch.tensor([L], dtype=torch.int32).cuda())
    kk = torch.stack([k[p] for p in used])
    vv = torch.stack([v[p] for p in used])
    ref, mag = dense.decode_paged(q, kk, vv, np.array([[0, 1, 2]]), [L], cfg.softmax_scale)
    dc.check_attention(out, ref, mag, dense.as_f64(q), dense.as_f64(kk), cfg.softmax_scale, L,
                       P_TWO_PARTS)
    # the append's and the prefill's addresses in the same buffer
    cu, sl = torch.tensor([0, 1]).cuda(), torch.tensor([L], dtype=torch.int32).cuda()
    new = dc.randn((1, 2 * G, d), 5)
    w = torch.zeros(8, device="cuda")
    msa.msa_rope_append_paged(cfg, None, new[:, :G], new[:, G:], w,
                              msa.paged_kv(k, v, torch.from_numpy(table).cuda()), cu, sl)
    assert torch.equal(k[64, (L - 1) % page], new[0, :G])
    assert torch.equal(v[64, (L - 1) % page], new[0, G:])
    kk[2, (L - 1) % page], vv[2, (L - 1) % page] = new[0, :G], new[0, G:]
    out = msa.msa_dense_prefill_paged(cfg, q, msa.paged_kv(k, v, torch.from_numpy(table).cuda()),
                                      cu, sl)
    ref, mag = dense.decode_paged(q, kk, vv, np.array([[0, 1, 2]]), [L], cfg.softmax_scale)
    dc.check_attention(out, ref, mag, dense.as_f64(q), dense.as_f64(kk), cfg.softmax_scale, L,
                       dc.HALF_BF16)
