"""Performance cases of the full-attention operators over packed and paged keys and values.

Four operators are measured:

* ``append``: rotate the queries and keys of new tokens by their positions and append the keys
  and values to a paged cache;
* ``prefill``: causal attention of whole prompts packed along the token axis, grouped heads;
* ``chunk``: causal attention of a few or many new tokens per sequence against the sequence's
  paged cache, which holds them already;
* ``decode``: attention of one new token per sequence over its paged cache.

A case is a dict of plain values.  Lengths of a batch are texts of numbers separated by blanks.
``own`` selects between the plain form (elementary torch operations in 32 bits, angles in 64)
and the calls a user makes of the package.
"""
import math

import torch

own = False

DEV = "cuda"


def _ints(text):
    return [int(x) for x in text.split()]


def listed():
    return [
        # one new token of each of 16 running requests, far into their contexts: the append in
        # front of a decode step (latency)
        dict(name="append_decode_step", op="append", H=64, G=8, d=128, rot=128, inter=0, page=64,
             new="1 " * 16, ctx="262143 1048575 4095 131071 70001 12 0 900 " * 2),
        # a whole 32K prompt written at once
        dict(name="append_prompt_32k", op="append", H=64, G=8, d=128, rot=128, inter=0, page=64,
             new="32768", ctx="0"),
        # chunks of several prompts of odd lengths, half of each head rotated, adjacent pairs
        dict(name="append_ragged_partial", op="append", H=12, G=4, d=64, rot=32, inter=1, page=16,
             new="1 777 130 2049 15 64", ctx="5 333 0 8191 17 100000"),
        # two short prompts (latency)
        dict(name="prefill_short", op="prefill", H=64, G=8, d=128, new="100 28"),
        # one 4K prompt of a small model
        dict(name="prefill_small_4k", op="prefill", H=4, G=2, d=64, new="4096"),
        # a packed batch of unequal prompts, five query heads to a key head
        dict(name="prefill_packed_ragged", op="prefill", H=20, G=4, d=128,
             new="1 17 8000 300 129 2048 5001 777 4096 128 63 1500"),
        # one 32K prompt
        dict(name="prefill_32k", op="prefill", H=64, G=8, d=128, new="32768"),
        # the next chunk of four long prompts over their caches
        dict(name="chunk_512", op="chunk", H=64, G=8, d=128, page=64, new="512 512 512 512",
             ctx="7680 16000 1000 30011"),
        # eight drafted tokens of each request checked at once over long caches: few rows
        dict(name="chunk_drafts", op="chunk", H=32, G=4, d=128, page=16, new="8 8 8 8",
             ctx="1001 65536 20000 7000"),
        # one request, a short cache (latency)
        dict(name="decode_one_4k", op="decode", H=64, G=8, d=128, page=16, lens="4097"),
        # a running batch of unequal requests
        dict(name="decode_ragged", op="decode", H=32, G=8, d=64, page=32,
             lens="1 33 16000 500 127 4096 9999 64 " * 6 + "12000 2 31 2500"),
        # sixteen requests of 256K tokens and one of 1M
        dict(name="decode_256k_1m", op="decode", H=64, G=8, d=128, page=128,
             lens="262144 " * 16 + "1048576"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _text(xs):
    return " ".join(str(x) for x in xs)


def draw(rng):
    """One more case of the same ranges."""
    op = rng.choice(["append", "prefill", "chunk", "decode"])
    d = rng.choice([64, 128])
    G = rng.choice([1, 2, 3, 4, 8])
    H = G * rng.choice([1, 2, 4, 5, 8, 16])
    c = dict(op=op, H=H, G=G, d=d)
    if op == "append":
        B = _log_int(rng, 1, 64)
        total = _log_int(rng, B, 32768)
        new = [max(1, int(total * rng.random() * 2 / B)) for _ in range(B)]
        c.update(rot=rng.choice([d, d // 2, 16]), inter=rng.choice([0, 1]),
                 page=rng.choice([16, 32, 64, 128, 256]), new=_text(new),
                 ctx=_text(_log_int(rng, 1, 1 << 20) - 1 for _ in range(B)))
    elif op == "prefill":
        B = _log_int(rng, 1, 16)
        c.update(new=_text(_log_int(rng, 1, max(2, 20000 // B)) for _ in range(B)))
    elif op == "chunk":
        B = _log_int(rng, 1, 4)
        c.update(page=rng.choice([16, 32, 64, 128, 256]),
                 new=_text(_log_int(rng, 1, 1024) for _ in range(B)),
                 ctx=_text(_log_int(rng, 1, 65536) - 1 for _ in range(B)))
    else:
        B = _log_int(rng, 1, 128)
        c.update(page=rng.choice([16, 32, 64, 128, 256]),
                 lens=_text(_log_int(rng, 1, max(16, 2000000 // B)) for _ in range(B)))
    return c


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _randn(shape, gen):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.bfloat16)


def _offsets(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _tables(lens, page, gen):
    """Block table [B][most pages] of pages in random order, and the pool's size."""
    need = [(n + page - 1) // page for n in lens]
    pool = max(1, sum(need))
    order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
    table = torch.zeros((len(lens), max(1, max(need))), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    op, H, G, d = case["op"], case["H"], case["G"], case["d"]
    s = dict(case=case, scale=1.0 / math.sqrt(d))
    if op == "append":
        new, ctx = _ints(case["new"]), _ints(case["ctx"])
        T, page, rot = sum(new), case["page"], case["rot"]
        # the fused projection's output: q, k, v are views of its rows
        qkv = _randn((T, (H + 2 * G) * d), gen)
        s["q"] = qkv[:, :H * d].view(T, H, d)
        s["k"] = qkv[:, H * d:(H + G) * d].view(T, G, d)
        s["v"] = qkv[:, (H + G) * d:].view(T, G, d)
        s["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device=DEV, dtype=torch.float64) / rot)
                         ).to(torch.float32)
        # only the pages that receive rows are kept apart: what lies before them is not read
        first = [c // page for c in ctx]
        last = [(c + n - 1) // page for c, n in zip(ctx, new)]
        need = [hi - lo + 1 for lo, hi in zip(first, last)]
        pool = sum(need)
        order = torch.randperm(pool, generator=gen, device=DEV).to(torch.int32)
        table = torch.zeros((len(new), max(last) + 1), dtype=torch.int32, device=DEV)
        at = 0
        for b, n in enumerate(need):
            table[b, first[b]:last[b] + 1] = order[at:at + n]
            at += n
        s["lens"] = [c + n for c, n in zip(ctx, new)]
    elif op == "prefill":
        new = _ints(case["new"])
        T = sum(new)
        s["q"], s["k"], s["v"] = _randn((T, H, d), gen), _randn((T, G, d), gen), _randn((T, G, d), gen)
    elif op == "chunk":
        new, ctx = _ints(case["new"]), _ints(case["ctx"])
        T, page = sum(new), case["page"]
        s["q"] = _randn((T, H, d), gen)
        s["lens"] = [c + n for c, n in zip(ctx, new)]
        table, pool = _tables(s["lens"], page, gen)
    else:
        s["lens"] = _ints(case["lens"])
        new, page = [1] * len(s["lens"]), case["page"]
        s["q"] = _randn((len(new), H, d), gen)
        table, pool = _tables(s["lens"], page, gen)
    s["new"], s["cu"] = new, _offsets(new)
    s["cu_dev"] = torch.tensor(s["cu"], dtype=torch.int64, device=DEV)
    if op != "prefill":
        s["seq_lens"] = torch.tensor(s["lens"], dtype=torch.int32, device=DEV)
        s["table"] = table
        s["k_cache"] = _randn((pool, page, G, d), gen)
        s["v_cache"] = _randn((pool, page, G, d), gen)
    if own:
        import block_sparse_long_branch_b200 as msa
        s["cfg"] = msa.config(H, G, d, d)
        if op != "prefill":
            s["kv"] = msa.paged_kv(s["k_cache"], s["v_cache"], s["table"])
        # the scratch a serving loop keeps from call to call
        which = dict(append=msa.OP_ROPE_APPEND, prefill=msa.OP_DENSE_PREFILL,
                     chunk=msa.OP_DENSE_PREFILL_PAGED, decode=msa.OP_DENSE_DECODE)[op]
        n = msa.msa_workspace_size(s["cfg"], which, s["q"].shape[0], len(new))
        s["ws"] = torch.empty(n, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------------------------
def _rotate(x, pos, inv_freq, inter):
    """x [T][heads][d] -> rotated, in 32 bits with the angles in 64."""
    r = 2 * inv_freq.shape[0]
    ang = pos.to(torch.float64)[:, None] * inv_freq.to(torch.float64)[None, :]
    c, sn = torch.cos(ang).float()[:, None, :], torch.sin(ang).float()[:, None, :]
    y = x.float().clone()
    if inter:
        a, b = y[..., 0:r:2].clone(), y[..., 1:r:2].clone()
        y[..., 0:r:2], y[..., 1:r:2] = a * c - b * sn, b * c + a * sn
    else:
        a, b = y[..., :r // 2].clone(), y[..., r // 2:r].clone()
        y[..., :r // 2], y[..., r // 2:r] = a * c - b * sn, b * c + a * sn
    return y.to(x.dtype)


def _attend(q, k, v, pos0, scale):
    """Causal attention of q [n][H][d] at positions pos0.. over k, v [L][G][d], in 32 bits."""
    n, H, d = q.shape
    L, G = k.shape[0], k.shape[1]
    if L == 0:
        return torch.zeros_like(q)
    hg = H // G
    out = torch.empty_like(q)
    rows = max(1, min(n, (1 << 28) // max(1, L * hg)))
    for g in range(G):
        kf, vf = k[:, g].float(), v[:, g].float()
        for a in range(0, n, rows):
            e = min(n, a + rows)
            m = min(L, pos0 + e)  # keys that some row of this chunk sees
            x = q[a:e, g * hg:(g + 1) * hg].float().reshape((e - a) * hg, d)
            sc = (x @ kf[:m].t()).mul_(scale).view(e - a, hg, m)
            hide = torch.arange(m, device=q.device)[None, :] > (
                torch.arange(a, e, device=q.device)[:, None] + pos0)
            sc.masked_fill_(hide[:, None, :], float("-inf"))
            sc.sub_(sc.amax(-1, keepdim=True)).exp_()
            den = sc.sum(-1, keepdim=True)
            o = (sc.view(-1, m) @ vf[:m]).view(e - a, hg, d) / den
            out[a:e, g * hg:(g + 1) * hg] = o.to(q.dtype)
    return out


def _gather(cache, table_row, L):
    page = cache.shape[1]
    n = (L + page - 1) // page
    return cache[table_row[:n].long()].reshape(n * page, *cache.shape[2:])[:L]


def _plain(s):
    c = s["case"]
    op, cu = c["op"], s["cu"]
    if op == "append":
        page = c["page"]
        pos = torch.cat([torch.arange(L - n, L, device=DEV) for n, L in zip(s["new"], s["lens"])])
        seq = torch.repeat_interleave(torch.arange(len(s["new"]), device=DEV),
                                      s["cu_dev"][1:] - s["cu_dev"][:-1])
        pg = s["table"][seq, pos // page].long()
        row = pos % page
        q = _rotate(s["q"], pos, s["inv_freq"], c["inter"])
        s["k_cache"][pg, row] = _rotate(s["k"], pos, s["inv_freq"], c["inter"])
        s["v_cache"][pg, row] = s["v"]
        return q, s["k_cache"], s["v_cache"]
    out = torch.empty_like(s["q"])
    for b, n in enumerate(s["new"]):
        a, e = cu[b], cu[b + 1]
        if op == "prefill":
            k, v, L = s["k"][a:e], s["v"][a:e], n
        else:
            L = s["lens"][b]
            k, v = _gather(s["k_cache"], s["table"][b], L), _gather(s["v_cache"], s["table"][b], L)
        out[a:e] = _attend(s["q"][a:e], k, v, L - n, s["scale"])
    return out


# ---------------------------------------------------------------------------------------------
def run(state):
    s = state
    if not own:
        return _plain(s)
    import block_sparse_long_branch_b200 as msa
    op = s["case"]["op"]
    if op == "append":
        q = msa.msa_rope_append_paged(s["cfg"], s["q"], s["k"], s["v"], s["inv_freq"], s["kv"],
                                      s["cu_dev"], s["seq_lens"],
                                      interleaved=bool(s["case"]["inter"]), workspace=s["ws"])
        return q, s["k_cache"], s["v_cache"]
    if op == "prefill":
        return msa.msa_dense_prefill_varlen(s["cfg"], s["q"], s["k"], s["v"], s["cu"],
                                            workspace=s["ws"])
    if op == "chunk":
        return msa.msa_dense_prefill_paged(s["cfg"], s["q"], s["kv"], s["cu_dev"], s["seq_lens"],
                                           workspace=s["ws"])
    return msa.msa_dense_decode_paged(s["cfg"], s["q"], s["kv"], s["seq_lens"], workspace=s["ws"])


def _visible(case):
    """Sum over the query tokens of the keys each one sees, and the keys of all sequences."""
    if case["op"] == "prefill":
        new = _ints(case["new"])
        ctx = [0] * len(new)
    elif case["op"] == "chunk":
        new, ctx = _ints(case["new"]), _ints(case["ctx"])
    else:
        lens = _ints(case["lens"])
        return sum(lens), sum(lens), len(lens)
    seen = sum(n * c + n * (n + 1) // 2 for n, c in zip(new, ctx))
    return seen, sum(new) + sum(ctx), sum(new)


def work(case):
    H, G, d = case["H"], case["G"], case["d"]
    if case["op"] == "append":
        T = sum(_ints(case["new"]))
        # every element read and written once; three operations per rotated element
        return {"bytes": 4 * T * (H + 2 * G) * d, "flops": 3 * T * (H + G) * case["rot"]}
    seen, keys, rows = _visible(case)
    return {"bytes": 4 * rows * H * d + 4 * keys * G * d, "flops": 4 * d * H * seen}


def exact(case, seed):
    """The definitions in 64 bits: rotation as a product of complex numbers, attention head by
    head with the scores of one head at a time."""
    s = prepare(case, seed)
    op, H, G, d = case["op"], case["H"], case["G"], case["d"]
    f64 = torch.float64
    if op == "append":
        page, rot = case["page"], case["rot"]
        kc, vc = s["k_cache"].to(f64), s["v_cache"].to(f64)
        qs = s["q"].to(f64)
        w = s["inv_freq"].to(f64)
        table = s["table"].cpu().tolist()
        for b, n in enumerate(s["new"]):
            a, e, p0 = s["cu"][b], s["cu"][b + 1], s["lens"][b] - n
            turn = torch.polar(torch.ones((), dtype=f64, device=DEV).expand(n, rot // 2),
                               torch.arange(p0, p0 + n, device=DEV, dtype=f64).outer(w))
            for src, heads in (("q", H), ("k", G)):
                x = s[src][a:e].to(f64)
                h = x[..., :rot]
                pair = (h.reshape(n, heads, rot // 2, 2) if case["inter"]
                        else h.reshape(n, heads, 2, rot // 2).transpose(2, 3)).contiguous()
                z = torch.view_as_real(torch.view_as_complex(pair) * turn[:, None, :])
                h = z if case["inter"] else z.transpose(2, 3)
                x = torch.cat([h.reshape(n, heads, rot), x[..., rot:]], -1)
                if src == "q":
                    qs[a:e] = x
                else:
                    kx = x
            done = 0
            while done < n:  # page by page
                p = p0 + done
                m = min(n - done, page - p % page)
                pg, r = table[b][p // page], p % page
                kc[pg, r:r + m] = kx[done:done + m]
                vc[pg, r:r + m] = s["v"][a + done:a + done + m].to(f64)
                done += m
        return qs, kc, vc
    out = torch.zeros((s["q"].shape[0], H, d), dtype=f64, device=DEV)
    for b, n in enumerate(s["new"]):
        a = s["cu"][b]
        if op == "prefill":
            L = n
            k, v = s["k"][a:a + n], s["v"][a:a + n]
        else:
            L, page = s["lens"][b], case["page"]
            ids = s["table"][b, torch.arange(L, device=DEV) // page].long() * page
            ids += torch.arange(L, device=DEV) % page
            k = s["k_cache"].view(-1, G, d).index_select(0, ids)
            v = s["v_cache"].view(-1, G, d).index_select(0, ids)
        if L == 0:
            continue
        key = torch.arange(L, device=DEV)
        for g in range(G):
            kd, vd = k[:, g].to(f64), v[:, g].to(f64)
            for h in range(g * (H // G), (g + 1) * (H // G)):
                step = max(1, (1 << 27) // L)
                for i in range(0, n, step):
                    j = min(n, i + step)
                    logit = (s["q"][a + i:a + j, h].to(f64) * s["scale"]) @ kd.T
                    seen = key[None] <= (L - n + torch.arange(i, j, device=DEV))[:, None]
                    out[a + i:a + j, h] = torch.softmax(
                        torch.where(seen, logit, torch.full_like(logit, -math.inf)), -1) @ vd
    return out
