"""Host-side checks of the full-attention entry points: sizes, refusals, the binding's argument
checks.  No call here reaches a kernel."""
import ctypes

import pytest
import torch

import block_sparse_long_branch_b200 as msa

P = ctypes.c_void_p(1 << 20)   # 16-byte aligned, never dereferenced: the calls are refused first
ODD = ctypes.c_void_p((1 << 20) + 2)
WS = ctypes.c_void_p(1 << 21)


def cfg(H=8, G=2, d=128, **kw):
    return msa.config(H, G, d, d, **kw)


def cache(**kw):
    base = dict(k=1 << 20, v=1 << 22, block_table=1 << 23, num_pages=4, page_stride=16 * 2 * 128,
                page_size=16, table_stride=8)
    base.update(kw)
    return msa._PagedKVStruct(**base)


def decode(c=None, q=P, kv=None, sl=P, B=2, out=P, ws=WS, n=1 << 30):
    kv = cache() if kv is None else kv
    return msa.load_library().msa_dense_decode_paged(ctypes.byref(c or cfg()), q, ctypes.byref(kv),
                                                     sl, B, out, ws, n, None)


def paged(c=None, q=P, kv=None, cu=P, sl=P, B=2, T=5, out=P, ws=WS, n=1 << 30):
    kv = cache() if kv is None else kv
    return msa.load_library().msa_dense_prefill_paged(ctypes.byref(c or cfg()), q, ctypes.byref(kv),
                                                      cu, sl, B, T, out, ws, n, None)


def varlen(cu, c=None, q=P, k=P, v=P, out=P, ws=WS, n=1 << 30):
    arr = (ctypes.c_int64 * len(cu))(*cu)
    return msa.load_library().msa_dense_prefill_varlen(ctypes.byref(c or cfg()), q, k, v, arr,
                                                       len(cu) - 1, out, ws, n, None)


def append(c=None, q=P, qs=1024, k=P, ks=256, v=P, vs=256, w=P, rot=128, kv=None, cu=P, sl=P, B=2,
           T=5, qo=P, ws=WS, n=256):
    kv = cache() if kv is None else kv
    return msa.load_library().msa_rope_append_paged(
        ctypes.byref(c or cfg()), q, qs, k, ks, v, vs, w, rot, 0, ctypes.byref(kv), cu, sl, B, T,
        qo, ws, n, None)


def calls_with(c):
    return [decode(c=c), paged(c=c), varlen([0, 5], c=c), append(c=c)]


@pytest.mark.parametrize("kw,status", [
    (dict(H=6, G=4), 1), (dict(d=96), 2), (dict(d=32), 2), (dict(H=258, G=2), 2),
    (dict(H=8192, G=8192), 2), (dict(scale=0.0), 1), (dict(scale=-1.0), 1),
    (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1), (dict(G=0), 1)])
def test_configurations(kw, status):
    base = dict(H=8, G=2, d=128)
    base.update(kw)
    G = base.pop("G")
    c = msa.config(base.pop("H"), 2, base.pop("d"), 128, **base)
    c.num_groups = G
    assert calls_with(c) == [status] * 4
    n = ctypes.c_size_t(0)
    for op in range(msa.OP_ROPE_APPEND, msa.OP_DENSE_DECODE + 1):
        assert msa.load_library().msa_workspace_size(ctypes.byref(c), op, 8, 8,
                                                     ctypes.byref(n)) == status


def test_group_ratios_that_the_sparse_calls_do_not_take():
    for H, G in ((40, 8), (3, 3), (128, 1), (33, 3)):
        for op in (msa.OP_ROPE_APPEND, msa.OP_DENSE_PREFILL, msa.OP_DENSE_PREFILL_PAGED,
                   msa.OP_DENSE_DECODE):
            assert msa.msa_workspace_size(cfg(H=H, G=G), op, 100, 100) >= 256


def test_pointers():
    for st in (decode(q=None), decode(out=None), decode(sl=None), decode(q=ODD), decode(out=ODD),
               decode(sl=ctypes.c_void_p((1 << 20) + 1)),
               paged(q=None), paged(out=None), paged(cu=None), paged(sl=None), paged(q=ODD),
               paged(cu=ctypes.c_void_p((1 << 20) + 4)),
               varlen([0, 5], q=None), varlen([0, 5], k=None), varlen([0, 5], v=None),
               varlen([0, 5], out=None), varlen([0, 5], k=ODD),
               append(k=None), append(v=None), append(w=None), append(cu=None), append(sl=None),
               append(q=None), append(qo=None), append(k=ODD), append(qo=ODD)):
        assert st == 1


def test_caches():
    for call in (decode, paged, append):
        for kw, st in ((dict(k=None), 1), (dict(v=None), 1), (dict(block_table=None), 1),
                       (dict(k=(1 << 20) + 8), 1), (dict(block_table=(1 << 20) + 2), 1),
                       (dict(num_pages=0), 1), (dict(table_stride=0), 1),
                       (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
                       (dict(page_size=0), 2),
                       (dict(page_stride=16 * 2 * 128 - 8), 1), (dict(page_stride=16 * 2 * 128 + 4), 1),
                       (dict(num_pages=2 ** 31), 2), (dict(page_stride=1 << 38), 2),
                       (dict(table_stride=(1 << 26) + 1), 2)):
            assert call(kv=cache(**kw)) == st, (call.__name__, kw)


def test_sizes_and_strides():
    assert decode(B=0) == 1 and paged(T=0) == 1 and paged(B=0) == 1 and append(T=0) == 1
    assert paged(T=1 << 26) == 2 and decode(B=1 << 24) == 2
    assert varlen([1, 5]) == 1 and varlen([0, 5, 3]) == 1 and varlen([0, 0]) == 1
    assert varlen([0, 1 << 26]) == 2
    assert append(qs=1016) == 1 and append(qs=1028) == 1 and append(ks=248) == 1
    assert append(vs=252) == 1
    assert append(rot=136) == 1 and append(rot=-16) == 1 and append(rot=24) == 2


def test_append_in_place_needs_packed_queries():
    assert append(qs=1032, q=P, qo=P, n=0) == 1
    # packed queries, one token, or another output: refused for the workspace only
    assert append(n=0) == 3 and append(qs=1032, T=1, n=0) == 3
    assert append(qs=1032, qo=ctypes.c_void_p(1 << 24), n=0) == 3


def test_workspaces():
    for call, op, T, B in ((decode, msa.OP_DENSE_DECODE, 2, 2),
                           (paged, msa.OP_DENSE_PREFILL_PAGED, 5, 2),
                           (append, msa.OP_ROPE_APPEND, 5, 2)):
        need = msa.msa_workspace_size(cfg(), op, T, B)
        assert call(n=need - 1) == 3 and call(ws=None) == 3
        assert call(ws=ctypes.c_void_p((1 << 21) + 8), n=need) == 3
    need = msa.msa_workspace_size(cfg(), msa.OP_DENSE_PREFILL, 5, 1)
    assert varlen([0, 5], n=need - 1) == 3 and varlen([0, 5], ws=None) == 3
    # more of anything never needs less
    size = lambda op, T, B: msa.msa_workspace_size(cfg(), op, T, B)
    assert size(msa.OP_DENSE_PREFILL, 128, 1) < size(msa.OP_DENSE_PREFILL, 4096, 1) <= \
        size(msa.OP_DENSE_PREFILL, 4096, 64)
    assert size(msa.OP_DENSE_DECODE, 4, 4) <= size(msa.OP_DENSE_DECODE, 4096, 4096)


def test_binding_refuses_tensors_off_the_device():
    t = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        msa.paged_kv(t, t, torch.zeros((1, 4), dtype=torch.int32))
    with pytest.raises(TypeError):
        msa.paged_kv(None, t, torch.zeros((1, 4), dtype=torch.int32))
    q = torch.zeros((5, 8, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        msa.msa_dense_prefill_varlen(cfg(), q, q[:, :2], q[:, :2], [0, 5])
    with pytest.raises(ValueError):
        msa.msa_dense_prefill_varlen(cfg(), q, q[:, :2], q[:, :2], [0, 4])
    with pytest.raises(ValueError):
        msa.msa_dense_decode_paged(cfg(), q, None, torch.zeros(5, dtype=torch.int32))
