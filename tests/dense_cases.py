"""Inputs and tolerances of the full-attention tests (packed and paged caches)."""
import numpy as np
import torch

from oracle import dense

HALF_BF16 = 2.0 ** -8   # half a step of bf16, relative
EPS32 = 2.0 ** -24      # half a step of fp32, relative


def randn(shape, seed, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=device).to(torch.bfloat16)


def offsets(lens):
    return [0] + np.cumsum(lens).tolist()


def pool(lens, page, G, d, seed, spare=2, fill=float("nan"), table_cols=None, side_by_side=False):
    """A cache of random rows for sequences of the given lengths: pages in random order, memory
    past each sequence's end and spare pages filled with `fill`.  Returns k, v, table (numpy too)."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    cols = table_cols or max(1, max(need, default=1))
    table = np.full((len(lens), cols), -1, dtype=np.int32)  # unread entries are not valid pages
    if side_by_side:
        both = torch.full((pages, 2, page, G, d), fill, dtype=torch.bfloat16, device="cuda")
        k, v = both[:, 0], both[:, 1]
    else:
        k = torch.full((pages, page, G, d), fill, dtype=torch.bfloat16, device="cuda")
        v = torch.full((pages, page, G, d), fill, dtype=torch.bfloat16, device="cuda")
    at = 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        for c, s in ((k, 1), (v, 2)):
            rows = randn((n, G, d), seed * 1000 + 2 * b + s)
            for i in range(need[b]):
                part = rows[i * page:(i + 1) * page]
                c[int(table[b, i]), :part.shape[0]] = part
    return k, v, torch.from_numpy(table).cuda(), table


def attention_tol(ref, mag, q, k, scale, keys, p_round):
    """Elementwise bound on |got - exact| of an attention output.

    * the bf16 output: half a step of the result;
    * each probability rounded once for the product with v: `p_round` of sum p|v| (HALF_BF16 for
      bf16; 2^-16 for two bf16 parts, whose second is rounded at 2^-8 of a 2^-8 remainder);
    * the scores: d products summed in fp32, each sum off by at most (d + 2) EPS32 of
      scale * |q| |k| (Cauchy-Schwarz), which moves every weight by that much relatively, and the
      normaliser as well: twice;
    * the sums over the keys, of v and of the normaliser: `keys` additions each at EPS32;
    * exp2 in fp32 (2 units in the last place) and the scaling of its argument, whose size is at
      most twice the largest score: 4 EPS32 times that, twice."""
    q, k = np.nan_to_num(q, posinf=0, neginf=0), np.nan_to_num(k, posinf=0, neginf=0)
    d = q.shape[-1]
    smax = scale * np.sqrt((q ** 2).sum(-1).max()) * np.sqrt((k ** 2).sum(-1).max())
    rel = p_round + 2 * (d + 2) * EPS32 * smax + 2 * keys * EPS32 + 16 * EPS32 * (smax + 1)
    return HALF_BF16 * np.abs(ref) * (1 + 2 * rel) + rel * (1 + HALF_BF16) * mag + 1e-30


def check_attention(got, ref, mag, q, k, scale, keys, p_round):
    got = got.double().cpu().numpy()
    tol = attention_tol(ref, mag, q, k, scale, keys, p_round)
    odd = ~np.isfinite(ref)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    np.testing.assert_array_equal(got[odd & ~np.isnan(ref)], ref[odd & ~np.isnan(ref)])
    err = np.where(odd, 0.0, np.abs(np.where(odd, 0.0, got) - np.where(odd, 0.0, ref)))
    bad = err > np.where(odd, np.inf, tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} elements off, worst "
                           f"{(err / np.where(odd, 1, tol)).max():.3g} of the tolerance, first at "
                           f"{np.argwhere(bad)[0].tolist()}")


def check_rotated(got, x, pos, w, interleaved):
    """Off by at most: half a step of bf16 of the result; and, of |x| + |y| of the pair (at most
    the largest pair sum of the row), three fp32 roundings, a sine and a cosine good to 2 units
    in the last place (2 EPS32 each of at most 1), and the angle's fraction of a turn rounded to
    fp32 at most 1 half turn: pi EPS32.  Together below 12 EPS32."""
    ref = dense.rope(x, pos, w, interleaved)
    xa = np.abs(dense.as_f64(x))
    size = 2 * xa.max(axis=-1, keepdims=True)
    tol = HALF_BF16 * np.abs(ref) + 12 * EPS32 * size * (1 + HALF_BF16)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-30)).max()
