"""Offsets of new tokens that descend or leave the range of the batch: recorded always, the sequence
skipped, and the valid sequences right, in the append and in the attention alike."""
import numpy as np
import pytest
import torch

from oracle import dense
from tests import dense_cases as dc

pytestmark = pytest.mark.gpu

H, G, D, PAGE, COLS = 4, 2, 64, 16, 8
BAD_INDEX = 0x201


@pytest.fixture(scope="module")
def msa(cuda_device):
    import block_sparse_long_branch_b200 as m
    m.load_library()
    return m


def valid(cu, T):
    """Which sequences are: offsets that ascend and stay within cu[0] .. cu[-1] and the T rows."""
    return [max(cu[0], 0) <= a <= e <= min(cu[-1], T) for a, e in zip(cu[:-1], cu[1:])]


def claims(cu, T):
    """How many valid sequences each row belongs to."""
    n = np.zeros(T, dtype=int)
    for (a, e), ok in zip(zip(cu[:-1], cu[1:]), valid(cu, T)):
        if ok:
            n[a:e] += 1
    return n


def batches():
    yield "two, the second one descends", [0, 100, 50], 100
    yield "last one descends", [0, 40, 60, 90, 60], 100
    yield "first one descends", [70, 0, 40, 60, 100], 100
    yield "leaves the range", [30, 60, 20, 60, 80], 100
    yield "passes the tokens given", [0, 40, 200, 60, 90], 100
    yield "middle one descends, rows of two sequences", [0, 40, 20, 60], 60
    for n in (33, 257, 600):
        yield f"{n}, the last one descends", list(range(n)) + [n - 20], n + 3
        yield f"{n}, one passes the tokens given", [*range(9), n + 50, *range(9, n)], n
        yield f"{n}, one descends, rows of two sequences", [*range(20), *range(10, n - 9)], n


CASES = {name: (cu, T) for name, cu, T in batches()}


def setup(cu, seed):
    """Lengths and a cache for every sequence, valid or not."""
    B = len(cu) - 1
    new = [max(e - a, 0) for a, e in zip(cu[:-1], cu[1:])]
    lens = [max(min(n + (7 * b) % 20, PAGE * COLS), n) for b, n in enumerate(new)]
    table = np.random.default_rng(seed).permutation(B * COLS).astype(np.int32).reshape(B, COLS)
    return new, lens, table


@pytest.mark.parametrize("name", CASES)
def test_append(msa, name):
    cu, T = CASES[name]
    B, ok = len(cu) - 1, valid(*CASES[name])
    new, lens, table = setup(cu, 3)
    cfg = msa.config(H, G, D, D)
    q, k, v = (dc.randn((T, n, D), i) for i, n in enumerate((H, G, G)))
    kc = torch.full((B * COLS, PAGE, G, D), 3.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    w = (10000.0 ** (-torch.arange(0, D, 2, dtype=torch.float64) / D)).float().cuda()
    out = torch.full_like(q, 7.0)
    ws = torch.full((256,), 0xFF, dtype=torch.uint8, device="cuda")
    msa.msa_rope_append_paged(cfg, q, k, v, w, msa.paged_kv(kc, vc, torch.from_numpy(table).cuda()),
                              torch.tensor(cu).cuda(), torch.tensor(lens, dtype=torch.int32).cuda(),
                              q_out=out, workspace=ws)
    assert msa.msa_get_device_error(ws) == BAD_INDEX
    n = claims(cu, T)
    assert (out[torch.from_numpy(n == 0)] == 7.0).all()
    rows, pos, pages = [], [], []
    for b in range(B):
        if ok[b]:
            p = np.arange(lens[b] - new[b], lens[b])
            rows += range(cu[b], cu[b + 1])
            pos += p.tolist()
            pages += table[b, p // PAGE].tolist()
    pos, pg = np.array(pos, dtype=np.int64), torch.tensor(pages, dtype=torch.int64)
    slot = torch.from_numpy(pos % PAGE)
    untouched = torch.ones(kc.shape[:2], dtype=torch.bool)
    untouched[pg, slot] = False
    assert (kc[untouched] == 3.0).all() and (vc[untouched] == 3.0).all()
    if rows and n.max() == 1:
        dc.check_rotated(out[rows], q[rows], pos, w, False)
        dc.check_rotated(kc[pg, slot], k[rows], pos, w, False)
        assert torch.equal(vc[pg, slot], v[rows])


@pytest.mark.parametrize("name", CASES)
def test_attention(msa, name):
    cu, T = CASES[name]
    B, ok = len(cu) - 1, valid(*CASES[name])
    new, lens, table = setup(cu, 5)
    cfg = msa.config(H, G, D, D)
    q = dc.randn((T, H, D), 11)
    k, v = (dc.randn((B * COLS, PAGE, G, D), 12 + i) for i in range(2))
    out = torch.full_like(q, 7.0)
    ws = torch.full((msa.msa_workspace_size(cfg, msa.OP_DENSE_PREFILL_PAGED, T, B),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    msa.msa_dense_prefill_paged(cfg, q, msa.paged_kv(k, v, torch.from_numpy(table).cuda()),
                                torch.tensor(cu).cuda(),
                                torch.tensor(lens, dtype=torch.int32).cuda(), out=out, workspace=ws)
    assert msa.msa_get_device_error(ws) == BAD_INDEX
    n = claims(cu, T)
    assert (out[torch.from_numpy(n == 0)] == 7.0).all()
    if n.max() > 1:
        return
    kd, vd, qd = dense.as_f64(k), dense.as_f64(v), dense.as_f64(q)
    ref, mag = np.full(q.shape, 7.0), np.zeros(q.shape)
    for b in range(B):
        if ok[b] and cu[b + 1] > cu[b]:
            a, e = cu[b], cu[b + 1]
            ref[a:e], mag[a:e] = dense.attend(qd[a:e], dense.paged_rows(kd, table[b], lens[b]),
                                              dense.paged_rows(vd, table[b], lens[b]),
                                              cfg.softmax_scale, lens[b] - new[b])
    dc.check_attention(out, ref, mag, qd, kd, cfg.softmax_scale, PAGE * COLS, dc.HALF_BF16)


@pytest.mark.parametrize("name", CASES)
def test_one_good_call_clears_the_word(msa, name):
    """The same sequences with offsets in order: nothing recorded, every row written."""
    cu, T = CASES[name]
    B = len(cu) - 1
    cu = sorted(min(c, T) for c in cu)
    new, lens, table = setup(cu, 7)
    cfg = msa.config(H, G, D, D)
    q, k, v = (dc.randn((T, n, D), i) for i, n in enumerate((H, G, G)))
    kc = torch.zeros((B * COLS, PAGE, G, D), dtype=torch.bfloat16, device="cuda")
    kv = msa.paged_kv(kc, kc.clone(), torch.from_numpy(table).cuda())
    args = torch.tensor(cu).cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
    w = torch.zeros(D // 2, device="cuda")
    ws = torch.full((msa.msa_workspace_size(cfg, msa.OP_DENSE_PREFILL_PAGED, T, B),), 0xFF,
                    dtype=torch.uint8, device="cuda")
    qr = msa.msa_rope_append_paged(cfg, q, k, v, w, kv, *args, workspace=ws)
    assert msa.msa_get_device_error(ws) == 0
    assert torch.equal(qr[cu[0]:cu[-1]], q[cu[0]:cu[-1]])
    msa.msa_dense_prefill_paged(cfg, qr, kv, *args, workspace=ws)
    assert msa.msa_get_device_error(ws) == 0
