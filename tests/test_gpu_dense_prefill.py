"""Full causal attention of packed prompts and of chunks over a paged cache, against fp64."""
import numpy as np
import pytest
import torch

from oracle import dense
from tests import dense_cases as dc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa(cuda_device):
    import block_sparse_long_branch_b200 as m
    m.load_library()
    return m


def run_varlen(msa, H, G, d, lens, seed=1, edit=None, scale=None):
    cu = dc.offsets(lens)
    T = cu[-1]
    q, k, v = (dc.randn((T, n, d), seed * 10 + i) for i, n in enumerate((H, G, G)))
    if edit:
        edit(q, k, v, cu)
    cfg = msa.config(H, G, d, d, scale=scale)
    ws = torch.full((msa.msa_workspace_size(cfg, msa.OP_DENSE_PREFILL, T, len(lens)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = msa.msa_dense_prefill_varlen(cfg, q, k, v, cu, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    sc = cfg.softmax_scale
    ref, mag = dense.prefill_varlen(q, k, v, cu, sc)
    dc.check_attention(out, ref, mag, dense.as_f64(q), dense.as_f64(k), sc, max(lens),
                       dc.HALF_BF16)
    return out


@pytest.mark.parametrize("H,G,d", [(4, 2, 64), (8, 1, 128), (5, 1, 128), (6, 6, 64), (3, 3, 128),
                                   (12, 4, 64), (128, 1, 64), (33, 3, 128)])
@pytest.mark.parametrize("lens", [[1], [1, 1, 2], [127, 128, 129], [300, 5, 0, 511]])
def test_varlen_shapes(msa, H, G, d, lens):
    run_varlen(msa, H, G, d, lens)


def test_varlen_many_sequences_in_two_passes(msa):
    """More sequences than one launch takes, most of them one token long."""
    rng = np.random.default_rng(3)
    lens = rng.integers(0, 4, size=1500).tolist()
    lens[1023], lens[1024] = 140, 150
    run_varlen(msa, 2, 1, 64, lens)


def test_varlen_long_prompt_of_few_heads_is_split(msa):
    """One head, 2600 tokens: 11 units, so the keys are split over the GPU and joined."""
    run_varlen(msa, 1, 1, 128, [2600])
    run_varlen(msa, 2, 2, 64, [1900, 3, 700])


def test_varlen_repeats_bit_for_bit(msa):
    a = run_varlen(msa, 1, 1, 64, [2000])
    b = run_varlen(msa, 1, 1, 64, [2000])
    assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [1e-3, 3.0])
def test_varlen_scales(msa, scale):
    """Flat weights, and weights on a few keys (the running maximum moves often)."""
    run_varlen(msa, 4, 2, 128, [700], scale=scale)


def test_varlen_rising_scores(msa):
    """Keys that grow along the sequence: every tile raises the maximum."""
    def edit(q, k, v, cu):
        n = k.shape[0]
        k[:] = (k.float() * torch.linspace(0.1, 6.0, n, device="cuda")[:, None, None]).to(k.dtype)
    run_varlen(msa, 4, 1, 64, [900], edit=edit)


@pytest.mark.parametrize("H,G,d,n", [(4, 2, 64, 400), (2, 2, 128, 300), (1, 1, 64, 1500)])
def test_varlen_odd_values_reach_only_the_tokens_that_see_them(msa, H, G, d, n):
    """NaN and infinities in v, NaN in k, in the middle of sequences: earlier tokens, other
    sequences and other columns keep their values."""
    def edit(q, k, v, cu):
        a = cu[1]
        v[a + n // 2, 0, 3] = float("nan")
        v[a + n // 2 + 5, 0, 7] = float("inf")
        v[a + n - 2, G - 1, 9] = float("-inf")
        v[a + n - 1, G - 1, 9] = float("inf")
        k[a + n - 3, 0, 1] = float("nan")
    run_varlen(msa, H, G, d, [77, n, 50], edit=edit)


def run_paged(msa, H, G, d, page, new, ctx, seed=1, pad=0, **pool_kw):
    lens = [c + n for c, n in zip(ctx, new)]
    k, v, table, tnp = dc.pool(lens, page, G, d, seed, **pool_kw)
    cu = dc.offsets(new)
    T = cu[-1] + pad
    q = dc.randn((T, H, d), seed * 10 + 7)
    cfg = msa.config(H, G, d, d)
    ws = torch.full((msa.msa_workspace_size(cfg, msa.OP_DENSE_PREFILL_PAGED, T, len(new)),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    out = torch.full((T, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    msa.msa_dense_prefill_paged(cfg, q, msa.paged_kv(k, v, table), torch.tensor(cu).cuda(),
                                torch.tensor(lens, dtype=torch.int32).cuda(), out=out, workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    ref, mag = dense.prefill_paged(q[:cu[-1]], k, v, tnp, cu, lens, cfg.softmax_scale)
    dc.check_attention(out[:cu[-1]], ref, mag, dense.as_f64(q), dense.as_f64(k),
                       cfg.softmax_scale, max(lens), dc.HALF_BF16)
    assert (out[cu[-1]:] == 5.0).all()  # rows behind the last sequence are left alone
    return out


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,G,d", [(8, 2, 64), (5, 1, 128), (2, 2, 128)])
def test_paged_chunks(msa, page, H, G, d):
    run_paged(msa, H, G, d, page, [1, 40, 0, 130, 17], [0, 300, 50, 95, 257])


def test_paged_few_rows_over_long_caches_are_split(msa):
    run_paged(msa, 8, 1, 128, 16, [3, 8], [5000, 2111])
    run_paged(msa, 16, 2, 64, 64, [1], [9001])


@pytest.mark.parametrize("H,G,d,page,new,ctx", [
    (16, 2, 64, 16, [700, 560, 3], [4200, 3600, 9000]),
    (16, 1, 128, 128, [900, 0, 520], [4100, 30, 4500]),
    (9, 3, 128, 32, [1300, 1000], [4200, 4600]),
])
def test_paged_units_that_do_not_fill_the_gpu_are_cut_into_even_shares(msa, H, G, d, page, new, ctx):
    """Units of tens of key tiles, too few for a CTA each and too many for two parts each: shares
    begin and end inside units, and several parts of a unit are joined."""
    a = run_paged(msa, H, G, d, page, new, ctx, pad=2)
    assert torch.equal(a, run_paged(msa, H, G, d, page, new, ctx, pad=2))


@pytest.mark.parametrize("H,G,d", [(8, 2, 64), (5, 1, 128)])
def test_paged_many_sequences_are_planned_on_the_device(msa, H, G, d):
    """More than 32 sequences: a planning kernel, units longest first, a long one split."""
    rng = np.random.default_rng(11)
    new = rng.integers(0, 12, size=45).tolist()
    ctx = rng.integers(0, 200, size=45).tolist()
    new[7], ctx[7] = 70, 9000
    new[40], ctx[40] = 300, 11
    run_paged(msa, H, G, d, 32, new, ctx, pad=3)


def test_paged_many_units_are_planned_on_the_device(msa):
    """More units than CTAs: several per CTA, none split."""
    run_paged(msa, 8, 8, 64, 128, [2600, 2100], [30, 0])


def test_paged_padded_batch_and_strided_pages(msa):
    run_paged(msa, 4, 2, 64, 32, [5, 9], [100, 0], pad=7, side_by_side=True, table_cols=11)


def test_paged_whole_prompt_equals_packed(msa):
    """A prompt in the cache with no earlier context is a packed prompt."""
    H, G, d, n = 8, 2, 128, 700
    q, k, v = (dc.randn((n, h, d), 70 + i) for i, h in enumerate((H, G, G)))
    cfg = msa.config(H, G, d, d)
    packed = msa.msa_dense_prefill_varlen(cfg, q, k, v, [0, n])
    page = 64
    np_ = -(-n // page)
    kc = torch.full((np_, page, G, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    kc.view(-1, G, d)[:n], vc.view(-1, G, d)[:n] = k, v
    kv = msa.paged_kv(kc, vc, torch.arange(np_, dtype=torch.int32, device="cuda")[None])
    paged = msa.msa_dense_prefill_paged(cfg, q, kv, torch.tensor([0, n]).cuda(),
                                        torch.tensor([n], dtype=torch.int32).cuda())
    assert torch.equal(packed, paged)


def test_paged_bad_entries_are_recorded(msa):
    """A page id outside the pool, and a sequence shorter than its new tokens: the error word says
    so, the other sequences are right, the bad sequence's rows are not written when skipped."""
    H, G, d, page = 4, 2, 64, 16
    lens, new = [40, 50, 3], [8, 8, 8]
    k, v, table, tnp = dc.pool([40, 50, 16], page, G, d, 5)
    cfg = msa.config(H, G, d, d)
    q = dc.randn((24, H, d), 55)
    ws = torch.empty(msa.msa_workspace_size(cfg, msa.OP_DENSE_PREFILL_PAGED, 24, 3),
                     dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 8, 16, 24]).cuda()
    out = torch.full((24, H, d), 5.0, dtype=torch.bfloat16, device="cuda")
    call = lambda ls, tb: msa.msa_dense_prefill_paged(
        cfg, q, msa.paged_kv(k, v, tb), cu, torch.tensor(ls, dtype=torch.int32).cuda(), out=out,
        workspace=ws)
    call(lens, table)  # sequence 2: 8 new tokens, length 3
    assert msa.msa_get_device_error(ws) == 0x201
    assert (out[16:] == 5.0).all()
    ref, mag = dense.prefill_paged(q[:16], k, v, tnp, [0, 8, 16], [40, 50], cfg.softmax_scale)
    dc.check_attention(out[:16], ref, mag, dense.as_f64(q), dense.as_f64(k), cfg.softmax_scale, 50,
                       dc.HALF_BF16)
    for bad in (-1, k.shape[0]):
        tb = table.clone()
        tb[1, 1] = bad
        call([40, 50, 16], tb)
        assert msa.msa_get_device_error(ws) == 0x201
        dc.check_attention(out[:8], ref[:8], mag[:8], dense.as_f64(q), dense.as_f64(k),
                           cfg.softmax_scale, 50, dc.HALF_BF16)
    call([40, 50, table.shape[1] * page + 1], table)  # past the block table's row
    assert msa.msa_get_device_error(ws) == 0x201
