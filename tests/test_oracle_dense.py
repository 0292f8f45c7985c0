"""The fp64 oracle of full attention and rotation, pinned by independent forms."""
import math

import numpy as np
import torch

import oracle
from oracle import dense


def rand(shape, seed):
    return np.random.default_rng(seed).standard_normal(shape)


def test_attend_is_softmax_attention():
    q, k, v = rand((7, 6, 16), 1), rand((20, 2, 16), 2), rand((20, 2, 16), 3)
    out, mag = dense.attend(q, k, v, 0.3, 13)
    t = lambda x: torch.from_numpy(x).transpose(0, 1)
    rep = lambda x: t(x).repeat_interleave(3, 0)
    mask = torch.arange(20)[None] <= torch.arange(13, 20)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(t(q), rep(k), rep(v), attn_mask=mask,
                                                           scale=0.3)
    np.testing.assert_allclose(out, ref.transpose(0, 1).numpy(), atol=1e-13)
    assert (mag + 1e-13 >= np.abs(out)).all()
    mag2 = dense.attend(q, k, np.abs(v), 0.3, 13)[0]
    np.testing.assert_allclose(mag, mag2, atol=1e-13)


def test_attend_is_the_sparse_oracle_when_every_block_is_kept():
    """With as many selected blocks as there are, block-sparse attention is full attention."""
    N, H, G, d = 300, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    bf = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)
    q, k, v, qi, ki = bf(N, H, d), bf(N, G, d), bf(N, G, d), bf(N, G, 64), bf(N, 64)
    sparse = oracle.prefill(q, k, v, qi, ki, block=128, top_k=4, scale=0.125)["out"]
    out, _ = dense.prefill_varlen(q, k, v, [0, N], 0.125)
    np.testing.assert_allclose(out, sparse, atol=1e-10)


def test_paged_and_packed_agree():
    lens, page = [5, 16, 33], 16
    k, v = [rand((n, 2, 8), 10 + n) for n in lens], [rand((n, 2, 8), 50 + n) for n in lens]
    table = np.array([[4, -1, -1], [0, -1, -1], [2, 5, 1]])
    kc, vc = np.full((6, page, 2, 8), np.nan), np.full((6, page, 2, 8), np.nan)
    for b, n in enumerate(lens):
        for p in range(n):
            kc[table[b, p // page], p % page] = k[b][p]
            vc[table[b, p // page], p % page] = v[b][p]
    q = rand((sum(lens), 4, 8), 9)
    cu = [0, 5, 21, 54]
    a = dense.prefill_varlen(q, np.concatenate(k), np.concatenate(v), cu, 0.4)[0]
    b = dense.prefill_paged(q, kc, vc, table, cu, lens, 0.4)[0]
    np.testing.assert_array_equal(a, b)
    last = [c - 1 for c in cu[1:]]
    d = dense.decode_paged(q[last], kc, vc, table, lens, 0.4)[0]
    np.testing.assert_allclose(d, a[last], atol=1e-14)
    assert (dense.decode_paged(q[:1], kc, vc, table[:1], [0], 0.4)[0] == 0).all()


def test_rope_turns_pairs_by_the_angle():
    w = np.array([1.0, 0.25, 1e-3])
    pos = np.array([0, 3, 1000])
    x = rand((3, 2, 10), 4)
    for il in (False, True):
        y = dense.rope(x, pos, w, il)
        np.testing.assert_array_equal(y[..., 6:], x[..., 6:])
        np.testing.assert_allclose(y[0], x[0], atol=0)
        for j in range(3):
            a, b = (2 * j, 2 * j + 1) if il else (j, j + 3)
            z = (x[..., a] + 1j * x[..., b]) * np.exp(1j * pos * w[j])[:, None]
            np.testing.assert_allclose(y[..., a] + 1j * y[..., b], z, atol=1e-12)


def test_rope_scores_depend_on_the_distance_only():
    w = np.array([1.0, 0.1, 0.01, 0.001])
    q, k = rand((1, 1, 8), 6), rand((1, 1, 8), 7)
    s = [float((dense.rope(q, [p], w) * dense.rope(k, [p - 5], w)).sum()) for p in (5, 77, 4096)]
    assert max(s) - min(s) < 1e-9 * math.sqrt(64)
