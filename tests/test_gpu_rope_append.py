"""Rotation of new queries and keys and the append to a paged cache, against fp64."""
import numpy as np
import pytest
import torch

from oracle import dense
from tests import dense_cases as dc
from tests.dense_cases import check_rotated

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def msa(cuda_device):
    import block_sparse_long_branch_b200 as m
    m.load_library()
    return m


def freqs(rot, base=10000.0):
    return (base ** (-torch.arange(0, rot, 2, dtype=torch.float64) / max(rot, 1))).float().cuda()


def run(msa, H, G, d, rot, interleaved, page, new, ctx, seed=1, fused=True, pad=0, in_place=False,
        side_by_side=False, with_q=True):
    cu = dc.offsets(new)
    T = cu[-1] + pad
    lens = [c + n for c, n in zip(ctx, new)]
    w = freqs(rot)
    if fused:
        qkv = dc.randn((T, (H + 2 * G) * d), seed)
        q = qkv[:, :H * d].view(T, H, d)
        k = qkv[:, H * d:(H + G) * d].view(T, G, d)
        v = qkv[:, (H + G) * d:].view(T, G, d)
    else:
        q, k, v = (dc.randn((T, n, d), seed + 3 * i) for i, n in enumerate((H, G, G)))
    # pages for the rows written; earlier table entries are not valid pages and must not matter
    first = [c // page for c in ctx]
    last = [(c + n - 1) // page if n else f - 1 for c, n, f in zip(ctx, new, first)]
    need = sum(l - f + 1 for f, l in zip(first, last))
    order = np.random.default_rng(seed).permutation(need + 1)
    table = np.full((len(new), max(max(last) + 1, 1)), -1, dtype=np.int32)
    at = 0
    for b, (f, l) in enumerate(zip(first, last)):
        table[b, f:l + 1] = order[at:at + l - f + 1]
        at += l - f + 1
    shape = (need + 1, 2, page, G, d) if side_by_side else (2, need + 1, page, G, d)
    both = torch.full(shape, 3.0, dtype=torch.bfloat16, device="cuda")
    kc, vc = (both[:, 0], both[:, 1]) if side_by_side else (both[0], both[1])
    cfg = msa.config(H, G, d, d)
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    kv = msa.paged_kv(kc, vc, torch.from_numpy(table).cuda())
    q_in = q.clone()
    q_out = q if in_place else torch.full((T, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    got = msa.msa_rope_append_paged(cfg, q if with_q else None, k, v, w, kv,
                                    torch.tensor(cu).cuda(),
                                    torch.tensor(lens, dtype=torch.int32).cuda(),
                                    interleaved=interleaved, q_out=q_out if with_q else None,
                                    workspace=ws)
    torch.cuda.synchronize()
    assert msa.msa_get_device_error(ws) == 0
    pos = np.concatenate([np.arange(L - n, L) for n, L in zip(new, lens)])
    if with_q:
        assert got.data_ptr() == q_out.data_ptr()
        check_rotated(got[:cu[-1]], q_in[:cu[-1]], pos, w, interleaved)
        rest = q_in[cu[-1]:] if in_place else torch.full_like(got[cu[-1]:], 7.0)
        assert torch.equal(got[cu[-1]:], rest)
    else:
        assert got is None
    # the rows written, and nothing else
    seq = np.repeat(np.arange(len(new)), new)
    pg, row = torch.from_numpy(table[seq, pos // page].astype(np.int64)), torch.from_numpy(pos % page)
    check_rotated(kc[pg, row], k[:cu[-1]], pos, w, interleaved)
    assert torch.equal(vc[pg, row], v[:cu[-1]])
    untouched = torch.ones(kc.shape[:2], dtype=torch.bool)
    untouched[pg, row] = False
    assert (kc[untouched] == 3.0).all() and (vc[untouched] == 3.0).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,G,d,rot", [(8, 2, 128, 128), (8, 2, 128, 64), (5, 5, 64, 64),
                                       (3, 1, 64, 16), (12, 4, 128, 112), (2, 1, 64, 0)])
def test_layouts(msa, H, G, d, rot, interleaved):
    run(msa, H, G, d, rot, interleaved, 16, [1, 33, 0, 16, 7], [0, 5, 9, 16, 1000])


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(msa, page):
    run(msa, 4, 2, 64, 64, False, page, [300, 1], [100, page - 1], side_by_side=True)


def test_far_positions(msa):
    """A million tokens in: the angle of the first pair is a million radians."""
    run(msa, 8, 2, 128, 128, False, 64, [3, 1, 2], [(1 << 20) - 3, 999_983, 777_777])
    run(msa, 8, 2, 128, 128, True, 256, [3, 1], [(1 << 26) - 3, 33_554_467])


def test_many_tokens_take_four_per_cta(msa):
    run(msa, 2, 1, 64, 32, True, 32, [1501, 2, 700], [3, 40, 0], pad=5)


def test_in_place_padding_and_keys_only(msa):
    run(msa, 4, 2, 64, 64, False, 16, [3, 9], [2, 30], fused=False, in_place=True, pad=4)
    run(msa, 4, 2, 128, 128, False, 16, [3, 9], [2, 30], with_q=False, pad=3)


def test_many_sequences(msa):
    rng = np.random.default_rng(8)
    new = rng.integers(0, 3, size=1100).tolist()
    ctx = rng.integers(0, 100, size=1100).tolist()
    run(msa, 2, 1, 64, 64, False, 16, new, ctx)


@pytest.mark.parametrize("B", [1, 31, 33, 256, 257, 600])
def test_bad_entries_anywhere_in_a_batch(msa, B):
    """One bad page id or length, in the first or last sequence, on a first, middle or last page:
    recorded, whatever the number of sequences; a good batch clears the word again."""
    H, G, d, page, cols = 2, 1, 64, 16, 8
    cfg = msa.config(H, G, d, d)
    new = [(5 * b) % 90 + 40 for b in range(B)]
    cu = dc.offsets(new)
    q, k, v = (dc.randn((cu[-1], n, d), i) for i, n in enumerate((H, G, G)))
    lens = [n + (7 * b) % 30 for b, n in enumerate(new)]
    lens = [min(n, page * cols) for n in lens]
    new = [min(n, l) for n, l in zip(new, lens)]
    table = np.arange(B * cols, dtype=np.int32).reshape(B, cols)
    kc = torch.zeros((B * cols, page, G, d), dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")

    def call(tb, ls, cu=cu):
        msa.msa_rope_append_paged(cfg, q, k, v, freqs(64),
                                  msa.paged_kv(kc, vc, torch.from_numpy(tb).cuda()),
                                  torch.tensor(cu).cuda(),
                                  torch.tensor(ls, dtype=torch.int32).cuda(), workspace=ws)
        return msa.msa_get_device_error(ws)
    assert call(table, lens) == 0
    for b in {0, B - 1}:
        first, last = (lens[b] - new[b]) // page, (lens[b] - 1) // page
        for p in {first, (first + last) // 2, last}:
            tb = table.copy()
            tb[b, p] = -1 if p == first else B * cols
            assert call(tb, lens) == 0x201
        for bad in (new[b] - 1, page * cols + 1):
            ls = list(lens)
            ls[b] = bad
            assert call(table, ls) == 0x201
        room = [page * cols] * B  # enough for any offsets
        kc[(B - 1) * cols:], vc[(B - 1) * cols:] = 0, 0
        assert call(table, room, cu[:-1] + [cu[-1] + 1]) == 0x201  # passes the tokens given
        assert not kc[(B - 1) * cols:].any() and not vc[(B - 1) * cols:].any()
        tb = table.copy()
        tb[b, last + 1:] = -1  # not a page of the sequence
        tb[b, :first] = -1
        assert call(tb, lens) == 0
    assert call(table, lens) == 0


def test_bad_entries_are_recorded_and_skipped(msa):
    H, G, d, page = 2, 1, 64, 16
    cfg = msa.config(H, G, d, d)
    q, k, v = (dc.randn((6, n, d), i) for i, n in enumerate((H, G, G)))
    w = freqs(64)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    cu = torch.tensor([0, 2, 4, 6]).cuda()

    def call(table, lens):
        kc = torch.full((4, page, G, d), 3.0, dtype=torch.bfloat16, device="cuda")
        vc = kc.clone()
        out = torch.full((6, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
        msa.msa_rope_append_paged(cfg, q, k, v, w,
                                  msa.paged_kv(kc, vc, torch.tensor(table, dtype=torch.int32).cuda()),
                                  cu, torch.tensor(lens, dtype=torch.int32).cuda(), q_out=out,
                                  workspace=ws)
        return kc, vc, out, msa.msa_get_device_error(ws)
    good = [[0], [1], [2]]
    kc, vc, ref, err = call(good, [2, 5, 16])
    assert err == 0
    for bad in (-1, 4, 2 ** 31 - 1):  # no such page: the queries are still rotated
        kc, vc, out, err = call([[0], [bad], [2]], [2, 5, 16])
        assert err == 0x201 and torch.equal(out, ref)
        assert (kc[1] == 3.0).all() and (kc[3] == 3.0).all()
        assert torch.equal(vc[2, 14:], v[4:])
    for bad in (1, -3, 17):  # fewer keys than new tokens; past the block table's row
        kc, vc, out, err = call(good, [2, bad, 16])
        assert err == 0x201
        assert torch.equal(out[:2], ref[:2]) and torch.equal(out[4:], ref[4:])
