"""Shared helpers of the paged-cache tests: batches over shuffled pages, the 64-bit definitions and the
error bounds that the tests hold the kernels to."""
from __future__ import annotations

import math

D = 128


def half_step(dtype):
    """Largest relative error of one rounding to the type."""
    import torch
    return torch.finfo(dtype).eps / 2


class Cache:
    """A page set with sequences of the given lengths on shuffled pages. Rows behind a sequence's
    last token and pages of no sequence hold NaN; table entries behind its pages are no page."""

    def __init__(self, kv, chunks, heads, page, dtype, seed=0, pad=0, spare=2, extra_cols=0, poison=True):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.kv, self.n, self.heads, self.page, self.dtype = g, list(kv), list(chunks), heads, page, dtype
        need = [(t + page - 1) // page for t in kv]
        pool = sum(need) + spare
        self.K = torch.randn((pool, heads, page, D), generator=g, device="cuda").to(dtype)
        self.V = torch.randn((pool, heads, page, D), generator=g, device="cuda").to(dtype)
        perm = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
        cols = max(need + [0]) + extra_cols
        self.table = torch.full((len(kv), cols), -7, dtype=torch.int32)
        used = []
        for s, m in enumerate(need):
            ids, perm = perm[:m], perm[m:]
            self.table[s, :m] = torch.tensor(ids, dtype=torch.int32)
            used.append(ids)
        if poison:
            keep = torch.zeros((pool, page), dtype=torch.bool)
            for s, ids in enumerate(used):
                for k, p in enumerate(ids):
                    keep[p, :max(0, min(page, kv[s] - k * page))] = True
            drop = ~keep.cuda()[:, None, :, None].expand_as(self.K)
            self.K[drop] = math.nan
            self.V[drop] = math.nan
        starts = [0]
        for c in chunks:
            starts.append(starts[-1] + c)
        self.starts, self.total = starts, starts[-1] + pad
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(list(kv), dtype=torch.int32, device="cuda")
        self.table = self.table.cuda()

    def randn(self, *shape, scale=1.0, dtype=None):
        import torch
        return (torch.randn(shape, generator=self.g, device="cuda") * scale).to(dtype or self.dtype)

    def handles(self, J, max_q=None):
        pages = J.jolt_pages_create(self.K, self.V)
        batch = J.jolt_batch(self.q_start, self.kv_len, self.table, self.total,
                             max(self.n + [0]) if max_q is None else max_q)
        return pages, batch

    def rows(self, s, h, X):
        """The first kv_len rows of one head of a page tensor, for sequence s."""
        m = (self.kv[s] + self.page - 1) // self.page
        return X[self.table[s, :m].long(), h].reshape(-1, D)[: self.kv[s]]


def attention_ref(c: Cache, Q, scale, causal, prefix_out=None, prefix_lse=None):
    """out, lse and their error bounds, in 64 bits, rows of no sequence NaN.

    The bound of out, with h = half a step of the type, A = sum_j w_j |v_j| (w the softmax weights) and
    ds a bound of a score's error: the weights enter a matrix product rounded to the type (h A), the
    result is rounded once (h |out|), scores are sums of 128 exact products held in 32 bits
    (ds = 130 2^-24 scale max_j sum |q k|, which changes a weight by 2 ds after normalisation) and
    the sums over up to 2^17 keys run in 32 bits in blocks (2^-19 A). lse: ds, the exponentials and their sum
    (2^-19), and its own rounding."""
    import torch
    N, Hq = Q.shape[0], Q.shape[1]
    g = Hq // c.heads
    out = torch.full((N, Hq, D), math.nan, dtype=torch.float64, device="cuda")
    lse = torch.full((N, Hq), math.nan, dtype=torch.float64, device="cuda")
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    h2 = half_step(Q.dtype)
    for s in range(len(c.kv)):
        n, T, r = c.n[s], c.kv[s], slice(c.starts[s], c.starts[s + 1])
        if n == 0:
            continue
        for h in range(c.heads):
            K, V = c.rows(s, h, c.K).double(), c.rows(s, h, c.V).double()
            for q in range(h * g, h * g + g):
                x = Q[r, q].double()
                z = x @ K.T * scale
                mag = (x.abs() @ K.abs().T * abs(scale)).amax(1) if T else torch.zeros(n, dtype=torch.float64, device="cuda")
                if causal:
                    last = T - n + torch.arange(n, device="cuda")
                    z = z.masked_fill(torch.arange(T, device="cuda")[None] > last[:, None], -math.inf)
                Vx, Ax = V, V.abs()
                if prefix_lse is not None:
                    z = torch.cat((z, prefix_lse[r, q].double()[:, None]), 1)
                if z.shape[1] == 0:
                    z = torch.full((n, 1), -math.inf, dtype=torch.float64, device="cuda")
                    Vx = Ax = torch.zeros((1, D), dtype=torch.float64, device="cuda")
                L = torch.logsumexp(z, 1)
                w = torch.exp(z - torch.where(torch.isinf(L), 0.0, L)[:, None])
                k = Vx.shape[0]
                o, A = w[:, :k] @ Vx, w[:, :k] @ Ax
                if prefix_out is not None:
                    po = prefix_out[r, q].double()
                    o, A = o + w[:, k:] * po, A + w[:, k:] * po.abs()
                ds = 130 * 2.0 ** -24 * mag
                out[r, q], lse[r, q] = o, L
                tol_o[r, q] = h2 * o.abs() + (h2 + 2 * ds[:, None] + 2.0 ** -19) * A + torch.finfo(Q.dtype).tiny
                tol_l[r, q] = ds + 2.0 ** -19 + 2.0 ** -23 * torch.where(torch.isinf(L), 0.0, L.abs())
    return out, lse, tol_o, tol_l


def check_attention(c: Cache, Q, out, lse, scale, causal, prefix_out=None, prefix_lse=None):
    """Every row of a sequence within its bound; rows of none as they were (the caller fills NaN)."""
    import torch
    ro, rl, to, tl = attention_ref(c, Q, scale, causal, prefix_out, prefix_lse)
    live = c.starts[-1]
    assert torch.isnan(out[live:].float()).all()
    err = (out[:live].double() - ro[:live]).abs()
    assert not torch.isnan(err).any(), "NaN or missing rows"
    bad = err > to[:live]
    assert not bad.any(), (int(bad.sum()), float((err / to[:live]).max()), bad.nonzero()[:4].tolist())
    if lse is not None:
        assert torch.isnan(lse[live:]).all()
        inf = torch.isinf(rl[:live])
        assert torch.equal(torch.isinf(lse[:live]), inf) and (lse[:live][inf] < 0).all()
        e = (lse[:live].double() - rl[:live])[~inf].abs()
        assert not (e > tl[:live][~inf]).any(), float((e / tl[:live][~inf]).max())


def norm_rope_ref(X, w, eps, positions, inv_freq, interleaved):
    """Rows normed and rotated in 64 bits, and the bound of the kernel's error: half a step of the
    type for the one rounding, and 48 steps of 2^-24 of the pair's magnitudes for the sum of 128
    squares in lanes of 8 (at most 12 roundings), root, quotient, two products, the sine and cosine
    (errors below 2^-22) and the rotation's three roundings."""
    import torch
    x = X.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
    y, mag = x.clone(), x.abs()
    if inv_freq is not None:
        h = inv_freq.numel()
        a = positions.double()[:, None, None] * inv_freq.double()
        u, v = (slice(0, 2 * h, 2), slice(1, 2 * h, 2)) if interleaved else (slice(0, h), slice(h, 2 * h))
        y[..., u] = x[..., u] * a.cos() - x[..., v] * a.sin()
        y[..., v] = x[..., v] * a.cos() + x[..., u] * a.sin()
        m = mag[..., u] + mag[..., v]
        mag[..., u] = m
        mag[..., v] = m
    t = X.dtype
    slack = 48 * 2.0 ** -24 * mag
    return y, half_step(t) * (y.abs() + slack) + slack + torch.finfo(t).tiny * half_step(t) * 2


def freqs(rope_dim, base=1.0e6):
    import torch
    return (base ** (-torch.arange(0, rope_dim, 2, dtype=torch.float64) / rope_dim)).float().cuda()
