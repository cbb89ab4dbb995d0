"""The growing cache on the GPU: norm and rotation of rows, append to pages and attention over them,
against the definitions in 64 bits (paged_common). Bounds are derived there."""
import ctypes
import math

import pytest

from paged_common import D, Cache, attention_ref, check_attention, freqs, half_step, norm_rope_ref

pytestmark = pytest.mark.gpu
SCALE = 1.0 / math.sqrt(D)


@pytest.fixture(scope="module")
def J():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from tensor_decomposition_b200 import build
    build.build()
    from tensor_decomposition_b200 import jolt
    return jolt


def _t(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float16


# ------------------------------------------------------------------ norm and rotation
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,hq,hk,norm,rope,inter,start", [
    (1, 1, 0, True, 128, False, 0),
    (1, 32, 8, True, 128, False, 131071),
    (3, 5, 1, False, 128, True, 77),
    (130, 40, 40, True, 64, False, 500000),
    (17, 7, 3, True, 16, True, 5),
    (9, 64, 8, True, 0, False, 0),
    (33, 12, 4, False, 96, False, 1 << 20),
    (700, 96, 8, True, 128, False, 9),          # more rows a token than a CTA takes at once
    (5000, 3, 2, True, 32, True, 1000),         # many tokens a CTA
])
def test_norm_rope(J, dtype, tokens, hq, hk, norm, rope, inter, start):
    import torch
    t = _t(dtype)
    g = torch.Generator(device="cuda").manual_seed(tokens * hq)
    x = (torch.randn((tokens, hq + 2 * hk, D), generator=g, device="cuda") * 1.7).to(t)   # a fused projection's rows
    x[0, 0] = 0                                                                          # a row of zeros
    Q, K = x[:, :hq], x[:, hq:hq + hk] if hk else None
    w = [(1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(t) if norm else None for _ in range(2)]
    pos = (start - torch.arange(tokens, device="cuda")).to(torch.int32)                  # below zero too
    f = freqs(rope) if rope else None
    Qo = torch.full((tokens, hq, D), math.nan, dtype=t, device="cuda")
    Ko = torch.full((tokens, hk, D), math.nan, dtype=t, device="cuda") if hk else None
    before = x.clone()
    J.jolt_qk_norm_rope(Q, Qo, K, Ko, positions=pos, inv_freq=f, q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=inter)
    assert torch.equal(x, before)
    for X, Y, wx in ((Q, Qo, w[0]), (K, Ko, w[1])):
        if X is None:
            continue
        ref, tol = norm_rope_ref(X, wx, 1e-5, pos, f, inter)
        err = (Y.double() - ref).abs()
        assert (err <= tol).all(), float((err / tol).max())
    # in place on the strided rows, the same bits
    J.jolt_qk_norm_rope(Q, Q, K, K, positions=pos, inv_freq=f, q_weight=w[0], k_weight=w[1], eps=1e-5, interleaved=inter)
    assert torch.equal(Q, Qo) and (K is None or torch.equal(K, Ko))
    assert torch.equal(x[:, hq + hk:], before[:, hq + hk:])


def test_norm_rope_of_nothing(J):
    import torch
    e = torch.empty((0, 8, D), dtype=torch.bfloat16, device="cuda")
    J.jolt_qk_norm_rope(e, e)


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv,chunks,heads,page,norm,rope,inter,own_pos,pad", [
    ([1], [1], 1, 16, True, 128, False, False, 0),
    ([16, 17, 40], [16, 1, 40], 8, 16, False, 128, False, True, 3),
    ([100, 5, 0, 64], [3, 5, 0, 64], 3, 48, True, 64, True, True, 0),
    ([2, 300], [5, 299], 2, 256, True, 128, False, False, 7),        # three tokens before the cache's begin: dropped
    ([33] * 300, [1] * 300, 2, 16, False, 0, False, False, 0),       # more sequences than a CTA has threads
    ([3000, 77, 2100], [2999, 5, 2050], 1, 32, True, 128, False, False, 9),   # many tokens a CTA, sequences meeting in one
    ([50, 9], [50, 2], 48, 16, True, 128, True, False, 0),           # more rows a token than a CTA takes at once
])
def test_append(J, dtype, kv, chunks, heads, page, norm, rope, inter, own_pos, pad):
    import torch
    t = _t(dtype)
    c = Cache(kv, chunks, heads, page, t, seed=len(kv), pad=pad, poison=False, extra_cols=1)
    x = c.randn(c.total, 3 * heads, D, scale=1.3)
    K, V = x[:, heads:2 * heads], x[:, 2 * heads:]
    if c.total > 1:
        V[1] = math.nan                          # values go out as they are, whatever they hold
    w = (1 + c.randn(D, scale=0.3, dtype=torch.float32)).to(t) if norm else None
    f = freqs(rope, 1e4) if rope else None
    pos = torch.full((c.total,), 0, dtype=torch.int32, device="cuda")
    place = {}
    for s in range(len(kv)):
        for i in range(chunks[s]):
            p = kv[s] - chunks[s] + i
            pos[c.starts[s] + i] = p + 100000 * own_pos
            if p >= 0:
                place[c.starts[s] + i] = (int(c.table[s, p // page]), p % page)
    Kp, Vp = c.K.clone(), c.V.clone()
    pages, batch = c.handles(J)
    J.jolt_paged_append(pages, batch, K, V, positions=pos if own_pos else None, inv_freq=f, k_weight=w, eps=1e-6,
                        interleaved=inter)
    J.jolt_pages_status(pages)
    ref, tol = norm_rope_ref(K, w, 1e-6, pos, f, inter)
    rows = list(place)
    pg, rw = (torch.tensor([place[r][k] for r in rows], device="cuda") for k in (0, 1))
    got = c.K[pg, :, rw].double()
    err = (got - ref[rows]).abs()
    assert (err <= tol[rows]).all(), float((err / tol[rows]).max())
    assert torch.equal(c.V[pg, :, rw].view(torch.int16), V[rows].contiguous().view(torch.int16))
    touched = torch.zeros(c.K.shape[:3], dtype=torch.bool, device="cuda")
    touched[pg, :, rw] = True
    assert torch.equal(c.K[~touched], Kp[~touched]) and torch.equal(c.V[~touched], Vp[~touched])
    # the same rows as jolt_qk_norm_rope gives
    Ko = torch.empty((c.total, heads, D), dtype=t, device="cuda")
    J.jolt_qk_norm_rope(K, Ko, positions=pos, inv_freq=f, q_weight=w, eps=1e-6, interleaved=inter)
    assert torch.equal(c.K[pg, :, rw], Ko[rows])


# ------------------------------------------------------------------ attention
def _attend(J, c, hq, causal=True, prefix=False, seed=0, max_q=None, scale=SCALE, lse=True, strided=False):
    import torch
    Q = c.randn(c.total, hq + (3 if strided else 0), D, scale=2.0)
    if strided:
        Q = Q[:, 2:2 + hq]
    out = torch.full((c.total, hq, D), math.nan, dtype=c.dtype, device="cuda")
    L = torch.full((c.total, hq), math.nan, device="cuda") if lse else None
    po = pl = None
    if prefix:
        po = c.randn(c.total, hq, D, dtype=torch.float32)
        pl = c.randn(c.total, hq, dtype=torch.float32) + math.log(max(c.kv + [1]))
        pl[0, 0] = -math.inf                     # a prefix without keys
    pages, batch = c.handles(J, max_q)
    J.jolt_paged_attention(pages, batch, Q, out, scale, causal=causal, lse=L, prefix_out=po, prefix_lse=pl)
    J.jolt_pages_status(pages)
    check_attention(c, Q, out, L, scale, causal, po, pl)
    return pages, batch, Q, out, L


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv,heads,g,page", [
    ([1], 1, 1, 16), ([63, 64, 65], 2, 4, 16), ([127, 128, 129, 1], 3, 5, 48), ([1000], 8, 4, 64),
    ([4097, 3, 700], 1, 16, 32), ([17] * 70, 2, 3, 16), ([2500] * 3, 40, 1, 128), ([333, 90], 2, 32, 16),
    ([20000], 1, 8, 256),
])
def test_single_tokens(J, dtype, kv, heads, g, page):
    _attend(J, Cache(kv, [1] * len(kv), heads, page, _t(dtype), seed=sum(kv)), heads * g)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kv,chunks,heads,g,page", [
    ([2], [2], 1, 1, 16), ([40, 41], [3, 4], 2, 4, 16), ([200, 5, 131], [5, 5, 2], 1, 8, 48),
    ([64], [64], 2, 1, 16), ([129, 256, 257], [129, 1, 130], 2, 4, 64), ([300, 4000], [256, 257], 1, 3, 128),
    ([700, 30], [513, 30], 2, 7, 32), ([2049], [2049], 1, 2, 256), ([128, 128, 1, 64], [33, 65, 1, 64], 8, 4, 16),
])
def test_chunks(J, dtype, causal, kv, chunks, heads, g, page):
    _attend(J, Cache(kv, chunks, heads, page, _t(dtype), seed=sum(kv)), heads * g, causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv,chunks", [([70, 1, 900], [1, 1, 1]), ([70, 6, 900, 300], [4, 6, 1, 200])])
def test_prefix_is_joined(J, dtype, kv, chunks):
    for lse in (True, False):
        _attend(J, Cache(kv, chunks, 2, 32, _t(dtype), seed=3, pad=2), 8, prefix=True, lse=lse)


@pytest.mark.parametrize("chunks", [[1, 1, 1, 1], [1, 0, 3, 9], [2, 0, 40, 300]])
@pytest.mark.parametrize("prefix", [False, True])
def test_rows_without_keys(J, chunks, prefix):
    """Unused slots (kv_len 0), chunks longer than the cache (rows before its begin see no key), no
    chunk, padded rows: out 0 and lse -inf without a prefix, the prefix itself with one."""
    import torch
    _attend(J, Cache([0, 5, 2, 200], chunks, 2, 16, torch.bfloat16, seed=9, pad=5), 8, prefix=prefix)


def test_strided_queries(J):
    import torch
    for chunks in ([1, 1], [9, 60]):
        _attend(J, Cache([100, 60], chunks, 2, 16, torch.bfloat16, seed=1), 8, strided=True)


def test_large_scores(J):
    """Scores of hundreds: weights that underflow, maxima that move a lot."""
    import torch
    for chunks in ([1, 1], [65, 140]):
        _attend(J, Cache([700, 513], chunks, 2, 16, torch.bfloat16, seed=1), 8, scale=3.0)
        _attend(J, Cache([700, 513], chunks, 2, 16, torch.bfloat16, seed=2), 8, scale=-1.0)
        _attend(J, Cache([700, 513], chunks, 2, 16, torch.bfloat16, seed=2), 8, scale=0.0)


def test_rising_scores(J):
    """Keys whose scores rise along the cache by hundreds, so that every block moves the maximum, and
    fall, so that none after the first does."""
    import torch
    for sign in (1.0, -1.0):
        for chunks in ([1], [130]):
            c = Cache([1500], chunks, 1, 16, torch.bfloat16, seed=4)
            ramp = torch.linspace(0, 40 * sign, 1500, device="cuda")
            for p in range(c.table.shape[1]):
                r = ramp[16 * p:16 * p + 16]
                c.K[c.table[0, p].long(), 0, :r.numel()] = (c.K[c.table[0, p].long(), 0, :r.numel()].float() * 0.1
                                                              + r[:, None]).to(torch.bfloat16)
            Q = (c.randn(c.total, 4, D).float().abs() * 0.3).to(torch.bfloat16)
            out = torch.full((c.total, 4, D), math.nan, dtype=torch.bfloat16, device="cuda")
            L = torch.full((c.total, 4), math.nan, device="cuda")
            pages, batch = c.handles(J)
            J.jolt_paged_attention(pages, batch, Q, out, SCALE, lse=L)
            check_attention(c, Q, out, L, SCALE, True)


def test_offsets_beyond_32_bits(J):
    """Pages beyond element 2^31 of the page tensors."""
    import torch
    pool, heads, page = 131072 + 40, 8, 16
    K = torch.zeros((pool, heads, page, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    assert K.numel() > 2 ** 31
    for chunks in ([1], [33]):
        c = Cache([500], chunks, heads, page, torch.bfloat16, seed=6, spare=0, poison=False)
        m = c.K.shape[0]
        K[-m:], V[-m:] = c.K, c.V
        Q = c.randn(c.total, 16, D)
        out = torch.full((c.total, 16, D), math.nan, dtype=torch.bfloat16, device="cuda")
        pages = J.jolt_pages_create(K, V)
        batch = J.jolt_batch(c.q_start, c.kv_len, c.table + (pool - m), c.total, max(c.n))
        J.jolt_paged_attention(pages, batch, Q, out, SCALE)
        check_attention(c, Q, out, None, SCALE, True)
        new = c.randn(c.total, heads, D)
        J.jolt_paged_append(pages, batch, new, new)
        assert torch.equal(K[int(c.table[0, 499 // page]) + pool - m, :, 499 % page], new[-1])


def test_repeatable(J):
    import torch
    for chunks in ([1, 1, 1], [70, 300, 3]):
        c = Cache([3000, 700, 9], chunks, 2, 16, torch.bfloat16, seed=11)
        pages, batch, Q, out, L = _attend(J, c, 8)
        for _ in range(3):
            o2, l2 = torch.zeros_like(out), torch.zeros_like(L)
            J.jolt_paged_attention(pages, batch, Q, o2, SCALE, lse=l2)
            assert torch.equal(o2, out) and torch.equal(l2, L)


def test_two_streams_at_once(J):
    """Calls on one page set on two streams at a time, as two programs would make them."""
    import torch
    c = Cache([3000, 700], [1, 1], 2, 16, torch.bfloat16, seed=12)
    d = Cache([3000, 700], [300, 260], 2, 16, torch.bfloat16, seed=12)
    d.K, d.V, d.table, d.kv_len = c.K, c.V, c.table, c.kv_len
    runs = [_attend(J, x, 8) for x in (c, d)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for k in range(20):
        for st, (pages, batch, Q, out, L) in zip(streams, runs):
            with torch.cuda.stream(st):
                o2 = torch.zeros_like(out)
                J.jolt_paged_attention(pages, batch, Q, o2, SCALE)
                outs.append((o2, out))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in outs)


def test_captured_and_replayed(J):
    """A generation step (rotate, append, attend) captured once, replayed with the batch's arrays
    rewritten between replays; two such graphs replayed on two streams at once."""
    import torch
    heads, g, page, t = 2, 4, 16, torch.bfloat16
    f = freqs(128)

    def make(seed, n):
        c = Cache([400, 30, 0], [n, n, 1], heads, page, t, seed=seed, extra_cols=1, poison=False, spare=8)
        c.table[0, 25], c.table[1, 2] = int(c.table.max()), int(c.table[0, 25])
        free = [p for p in range(c.K.shape[0]) if p not in c.table.unique().tolist()]
        c.table[0, 25], c.table[1, 2], c.table[1, 3], c.table[2, 0] = free[0], free[1], free[2], free[3]
        x = c.randn(c.total, (g + 2) * heads, D)
        q = torch.empty((c.total, g * heads, D), dtype=t, device="cuda")
        out = torch.zeros((c.total, g * heads, D), dtype=t, device="cuda")
        pos = torch.arange(c.total, device="cuda", dtype=torch.int32)
        pages, batch = c.handles(J, max_q=n)

        def step():
            J.jolt_qk_norm_rope(x[:, :g * heads], q, positions=pos, inv_freq=f)
            J.jolt_paged_append(pages, batch, x[:, g * heads:(g + 1) * heads], x[:, (g + 1) * heads:], positions=pos,
                                inv_freq=f)
            J.jolt_paged_attention(pages, batch, q, out, SCALE)
        return c, x, q, out, pages, step

    sets = [make(1, 1), make(2, 20)]
    graphs, side = [], torch.cuda.Stream()
    for c, x, q, out, pages, step in sets:
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in sets]
    for it in range(4):
        for c, x, q, out, pages, step in sets:
            c.kv = [400 + it, 30 + it, 0 if it < 2 else 1]
            c.kv_len.copy_(torch.tensor(c.kv, dtype=torch.int32))
            x.copy_(c.randn(*x.shape))
        torch.cuda.synchronize()
        for _ in range(5):
            for gr, st in zip(graphs, streams):
                with torch.cuda.stream(st):
                    gr.replay()
        torch.cuda.synchronize()
        for c, x, q, out, pages, step in sets:
            J.jolt_pages_status(pages)
            check_attention(c, q, out, None, SCALE, True)


def test_a_run_of_them_together(J):
    """A prompt in two chunks and single tokens after it, through all three entry points, against
    attention over the exact keys and values (the pages hold the rounded rotated keys, so the
    reference attends over what the pages hold; what they hold is checked by the append's tests)."""
    import torch
    heads, g, page, t = 2, 3, 16, torch.float16
    chunks = [100, 37, 1, 1, 1]
    c = Cache([sum(chunks)], [1], heads, page, t, seed=21)
    pages = J.jolt_pages_create(c.K, c.V)
    f, at = freqs(64, 1e4), 0
    w = (1 + c.randn(D, scale=0.2, dtype=torch.float32)).to(t)
    for n in chunks:
        at += n
        x = c.randn(n, (g + 2) * heads, D)
        pos = torch.arange(at - n, at, device="cuda", dtype=torch.int32)
        c.kv, c.n, c.starts, c.total = [at], [n], [0, n], n
        c.q_start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        c.kv_len = torch.tensor([at], dtype=torch.int32, device="cuda")
        batch = J.jolt_batch(c.q_start, c.kv_len, c.table, n, n)
        q = torch.empty((n, g * heads, D), dtype=t, device="cuda")
        out, L = torch.full_like(q, math.nan), torch.full((n, g * heads), math.nan, device="cuda")
        J.jolt_qk_norm_rope(x[:, :g * heads], q, positions=pos, inv_freq=f, q_weight=w)
        J.jolt_paged_append(pages, batch, x[:, g * heads:(g + 1) * heads], x[:, (g + 1) * heads:], inv_freq=f, k_weight=w)
        J.jolt_paged_attention(pages, batch, q, out, SCALE, lse=L)
        check_attention(c, q, out, L, SCALE, True)
    J.jolt_pages_status(pages)


@pytest.mark.parametrize("n", [1, 7])
def test_compressed_prefix_and_paged_tail(J, n):
    """A context whose first tokens are a compressed stream and the rest in pages: one layer's attention over
    both, against softmax over the stream's reconstruction and the pages together, in 64 bits.

    The stream's part is held to 1e-4 of the largest output and 1e-4 in its log-sum-exp as in the tests
    of jolt_attention (32-bit sums of exact values); what the pages add is within attention_ref's
    bound. A shift d of the prefix's log-sum-exp moves a row by at most d times twice its largest value."""
    import numpy as np
    import torch

    import synth
    from gpu_common import gpu_encode, host
    from oracle import attention as oa
    from oracle import stream as ostream
    from oracle.jolt import decode_lt
    from oracle.numerics import rotation_matrix
    cfg = synth.config(1, layers=3, tokens=300, heads=4, seed=1709, groups=3)
    K, V = synth.gen_cache_numpy(cfg)
    _, st, _, _ = gpu_encode(cfg, K, V, synth.bf16_bytes(cfg) // 2, "sketch")
    layer, hq, tail = 1, 8, 45
    c = Cache([tail], [n], 4, 16, torch.bfloat16, seed=5)
    Q = c.randn(n, hq, D, scale=0.7)
    po = torch.full((n, hq, D), math.nan, device="cuda")
    pl = torch.full((n, hq), math.nan, device="cuda")
    out = torch.full((n, hq, D), math.nan, dtype=torch.bfloat16, device="cuda")
    L = torch.full((n, hq), math.nan, device="cuda")
    pages, batch = c.handles(J)
    J.jolt_attention_lse(st, layer, Q, po, pl, SCALE)
    J.jolt_paged_attention(pages, batch, Q, out, SCALE, lse=L, prefix_out=po, prefix_lse=pl)
    J.jolt_pages_status(pages)
    # the same rows as the entry point for all layers gives
    whole = torch.zeros((3, hq, n, D), dtype=torch.bfloat16, device="cuda")
    whole[layer] = Q.transpose(0, 1)
    ow = torch.zeros(whole.shape, device="cuda")
    J.jolt_attention(st, whole, ow, SCALE)
    assert torch.equal(ow[layer].transpose(0, 1), po)
    ost = ostream.parse(J.jolt_stream_to_host(st), lts={2 * layer, 2 * layer + 1})
    Pi = rotation_matrix(ost.seed, ost.D, ost.rotation)
    Kh, Vh = (decode_lt(ost, 2 * layer + k, Pi) for k in (0, 1))
    q = host(Q)
    for h in range(hq):
        kv = oa.kv_head_of(h, hq, 4)
        kt, vt = host(c.rows(0, kv, c.K)), host(c.rows(0, kv, c.V))
        for i in range(n):
            see = tail - n + i + 1
            sp, sq = SCALE * Kh[kv] @ q[i, h], SCALE * kt[:see] @ q[i, h]
            ref_l = np.log(np.exp(sp).sum())
            assert abs(float(pl[i, h]) - ref_l) <= 1e-4 * (1 + abs(ref_l))
            s = np.concatenate([sp, sq])
            p = np.exp(s - s.max())
            ref = (p[:, None] * np.concatenate([Vh[kv], vt[:see]])).sum(0) / p.sum()
            A = (p[:, None] * np.abs(np.concatenate([Vh[kv], vt[:see]]))).sum(0) / p.sum()
            big = max(np.abs(Vh[kv]).max(), np.abs(vt[:see]).max())
            u = half_step(torch.bfloat16)
            tol = u * np.abs(ref) + (u + 2.0 ** -14) * A + (1e-4 + 2e-4) * big + 1e-6
            got = host(out)[i, h]
            assert (np.abs(got - ref) <= tol).all(), float((np.abs(got - ref) / tol).max())
            assert abs(float(L[i, h]) - (np.log(p.sum()) + s.max())) <= 2e-4 * (1 + abs(ref_l))
    with pytest.raises(J.JoltError):
        J.jolt_attention_lse(st, 3, Q, po, pl, SCALE)
    with pytest.raises(ValueError):
        J.jolt_attention_lse(st, 0, Q, po, pl[:, :1], SCALE)


# ------------------------------------------------------------------ what the device refuses
@pytest.mark.parametrize("chunks", [[1, 1, 1], [3, 70, 5]])
def test_bad_bounds_and_pages_are_skipped_and_reported(J, chunks):
    import torch
    c = Cache([100, 200, 50], chunks, 2, 16, torch.bfloat16, seed=2, poison=False)
    Q = c.randn(c.total, 8, D)
    good = torch.full((c.total, 8, D), math.nan, dtype=torch.bfloat16, device="cuda")
    pages, batch = c.handles(J)
    J.jolt_paged_attention(pages, batch, Q, good, SCALE)
    J.jolt_pages_status(pages)
    K0, V0 = c.K.clone(), c.V.clone()
    kv = x = c.randn(c.total, 2, D)
    ref, _, tol, _ = attention_ref(c, Q, SCALE, True)
    assert ((good.double() - ref).abs() <= tol).all()

    def expect(text, rows):
        """The call reports `text`; the rows of the other sequences are right; then all is well again."""
        out = torch.full_like(good, math.nan)
        J.jolt_paged_attention(pages, batch, Q, out, SCALE)
        with pytest.raises(J.JoltError) as e:
            J.jolt_pages_status(pages)
        assert text in str(e.value) and e.value.status == 1
        J.jolt_pages_status(pages)
        for s in range(3):
            r = slice(c.starts[s], c.starts[s + 1])
            if s not in rows:   # not the same bits: a skipped sequence shifts where the others are divided
                assert ((out[r].double() - ref[r]).abs() <= tol[r]).all()
        J.jolt_paged_append(pages, batch, x, kv)
        with pytest.raises(J.JoltError):
            J.jolt_pages_status(pages)
        c.K.copy_(K0), c.V.copy_(V0)
        return out

    for bad in (-1, 13 + 7 + 4 + 2, 2 ** 31 - 1):          # no page of the set (its pages: 7 + 13 + 4 and 2 spare)
        t = c.table.clone()
        c.table[1, (200 - 1) // 16] = bad
        out = expect("page", {1})
        assert not torch.isnan(out.float()).any()
        c.table.copy_(t)
    for bad in (-5, 16 * c.table.shape[1] + 1, 2 ** 31 - 1):
        c.kv_len[1] = bad
        out = expect("kv_len", {1})
        assert torch.isnan(out[c.starts[1]:c.starts[2]].float()).all()     # skipped
        c.kv_len[1] = 200
    c.q_start[3] = c.total + 1
    expect("q_start", {2})
    c.q_start[3] = c.total
    c.q_start[0] = -1
    expect("q_start", {0})
    c.q_start[0] = 0
    small = J.jolt_batch(c.q_start, c.kv_len, c.table, c.total, max(chunks) - 1)
    out = torch.full_like(good, math.nan)
    J.jolt_paged_attention(pages, small, Q, out, SCALE)
    with pytest.raises(J.JoltError):
        J.jolt_pages_status(pages)


def test_binding_refuses(J):
    import torch
    c = Cache([100], [1], 2, 16, torch.bfloat16, poison=False)
    pages, batch = c.handles(J)
    Q, out = c.randn(1, 8, D), torch.empty((1, 8, D), dtype=torch.bfloat16, device="cuda")
    ok = dict(pages=pages, batch=batch, Q=Q, out=out, scale=SCALE)
    pre = torch.zeros((1, 8, D), device="cuda")
    for kw in (dict(Q=Q.half()), dict(Q=Q[:, :, :64]), dict(out=out.float()), dict(Q=Q.cpu()), dict(out=out[:, :4]),
               dict(Q=Q.transpose(1, 2).contiguous().transpose(1, 2)), dict(lse=torch.zeros((1, 7), device="cuda")),
               dict(prefix_out=pre.half(), prefix_lse=pre[..., 0].contiguous())):
        with pytest.raises(ValueError):
            J.jolt_paged_attention(**{**ok, **kw})
    with pytest.raises(J.JoltError):                       # a prefix without its log-sum-exp
        J.jolt_paged_attention(**ok, prefix_out=pre)
    with pytest.raises(J.JoltError):                       # 7 query heads over 2 KV heads
        J.jolt_paged_attention(pages, batch, Q[:, :7], out[:, :7].contiguous(), SCALE)
    odd = torch.empty(D * 8 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(1, 8, D)
    with pytest.raises(J.JoltError) as e:                  # rows off their 16-byte boundaries
        J.jolt_paged_attention(pages, batch, odd, out, SCALE)
    assert "16-byte" in str(e.value)
    with pytest.raises(J.JoltError):
        J.jolt_qk_norm_rope(odd, odd)
    with pytest.raises(J.JoltError):                       # 24 features cannot be rotated
        J.jolt_qk_norm_rope(Q, out, positions=c.kv_len, inv_freq=freqs(24))
    with pytest.raises(ValueError):
        J.jolt_qk_norm_rope(Q, out, inv_freq=freqs(32))
    with pytest.raises(ValueError):
        J.jolt_pages_create(c.K.float(), c.V.float())
    with pytest.raises(J.JoltError) as e:
        J.jolt_pages_create(c.K[:, :, :8].contiguous(), c.V[:, :, :8].contiguous())
    assert e.value.status == 9
    with pytest.raises(ValueError):
        J.jolt_batch(c.q_start.long(), c.kv_len, c.table, 1, 1)
    with pytest.raises(ValueError):
        J.jolt_batch(c.q_start, c.kv_len[:0], c.table, 1, 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("n", [17, 32, 127, 128, 129, 257, 300, 384])
def test_row_blocks_of_every_fill(J, dtype, n):
    """Chunks whose last block of rows holds one to 256 of them, over one key tile, two, three and many."""
    _attend(J, Cache([n, n + 100, n + 256, n + 5000], [n] * 4, 1, 16, _t(dtype), seed=n), 1)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("seqs,heads,g,n,kv", [
    (2, 8, 4, 5, 300),        # 16 items: clusters
    (3, 8, 4, 8, 700),        # 24 items: shares
    (40, 2, 16, 2, 90),       # 80 items, few keys: the kernel for many rows
    (33, 2, 5, 4, 9000),      # 66 items, many keys: shares
])
def test_seventeen_to_thirty_two_rows(J, dtype, seqs, heads, g, n, kv):
    c = Cache([max(n, kv - 7 * s) for s in range(seqs)], [n - s % 2 for s in range(seqs)], heads, 16, _t(dtype), seed=n, pad=3)
    _attend(J, c, heads * g, max_q=n, prefix=True)


@pytest.mark.parametrize("chunk,g", [(1, 2), (3, 12), (9, 8)])
def test_more_sequences_than_threads(J, chunk, g):
    """Batches that the kernels' threads have to go over more than once, long and short ones mixed."""
    import torch
    kv = [1 + (s * 37) % 150 for s in range(700)]
    kv[650], kv[3] = 4000, 0
    c = Cache(kv, [min(chunk, max(1, t)) for t in kv], 1, 16, torch.bfloat16, seed=chunk)
    _attend(J, c, g, max_q=chunk)


def test_one_page_for_two_sequences(J):
    """Sequences that share pages of a common beginning."""
    import torch
    for chunks in ([1, 1], [40, 9]):
        c = Cache([130, 100], chunks, 2, 16, torch.bfloat16, seed=8)
        c.table[1, :5] = c.table[0, :5]
        _attend(J, c, 8)


def test_captured_without_a_first_call():
    """The first calls of a process may be made while a graph is captured."""
    import subprocess
    import sys
    code = """
import torch, math, sys
sys.path.insert(0, 'tests')
from paged_common import Cache, check_attention
from tensor_decomposition_b200 import jolt as J
c = Cache([900, 40], [1, 1], 8, 16, torch.bfloat16, seed=1)
d = Cache([900, 40], [70, 9], 8, 16, torch.bfloat16, seed=1)
for x in (c, d):
    Q = x.randn(x.total, 32, 128)
    out = torch.full((x.total, 32, 128), math.nan, dtype=torch.bfloat16, device='cuda')
    pages, batch = x.handles(J)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        J.jolt_qk_norm_rope(Q, Q)
        J.jolt_paged_attention(pages, batch, Q, out, 0.1)
    g.replay()
    torch.cuda.synchronize()
    J.jolt_pages_status(pages)
    check_attention(x, Q, out, None, 0.1, True)
print('fine')
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


def test_results_do_not_depend_on_unread_memory(J):
    """The same call over pages whose unused rows, unused pages and table entries hold other things."""
    import torch
    for chunks in ([1, 1, 1], [5, 5, 5], [70, 3, 129]):
        outs = []
        for fill in (float("nan"), 0.0, float("inf")):
            c = Cache([200, 77, 129], chunks, 2, 16, torch.bfloat16, seed=14)
            c.K[torch.isnan(c.K)] = fill
            c.V[torch.isnan(c.V)] = fill
            outs.append(_attend(J, c, 8)[3])
        assert all(torch.equal(outs[0], o) for o in outs[1:])


@pytest.mark.parametrize("prefix", [False, True])
@pytest.mark.parametrize("kv,chunks,heads,g", [
    ([300, 40], [1, 1], 2, 4),               # clusters
    ([30000, 40], [1, 1], 2, 4),             # up to 8 rows, items in many shares
    ([30000, 40], [3, 2], 2, 4),             # up to 16
    ([30000, 40], [7, 2], 2, 4),             # up to 32
    ([30000, 40], [30, 20], 2, 4),           # a chunk of half a block, in many shares
    ([30000, 140], [100, 140], 2, 4),        # whole blocks, in many shares
    ([256] * 80, [256] * 80, 2, 2),          # many more blocks than CTAs
])
def test_queries_that_are_no_numbers(J, kv, chunks, heads, g, prefix):
    """Such a row's output and log-sum-exp are none either, however its keys are divided; the other rows'
    are as they should be."""
    import torch
    c = Cache(kv, chunks, heads, 16, torch.bfloat16, seed=5)
    pages, batch, Q, good, L0 = _attend(J, c, heads * g)
    po = pl = None
    if prefix:
        po, pl = c.randn(c.total, heads * g, D, dtype=torch.float32), c.randn(c.total, heads * g, dtype=torch.float32)
    rows, hd = [0, c.total // 2, c.total - 1], [0, 3, heads * g - 1]
    bad = Q.clone()
    bad[rows, hd, 77] = math.nan
    out, L = torch.zeros_like(good), torch.zeros_like(L0)
    J.jolt_paged_attention(pages, batch, bad, out, SCALE, lse=L, prefix_out=po, prefix_lse=pl)
    J.jolt_pages_status(pages)
    assert torch.isnan(out[rows, hd].float()).all() and torch.isnan(L[rows, hd]).all()
    J.jolt_paged_attention(pages, batch, Q, good, SCALE, lse=L0, prefix_out=po, prefix_lse=pl)
    out[rows, hd], L[rows, hd] = good[rows, hd], L0[rows, hd]
    check_attention(c, Q, out, L, SCALE, True, po, pl)


def test_sizes_that_pass_32_bits(J):
    """max_q bounds the chunks from above, however far; what the kernels could not count is refused."""
    import ctypes
    import torch
    _attend(J, Cache([900, 40], [1, 1], 2, 16, torch.bfloat16, seed=2), 8, max_q=2 ** 31 - 1)
    c = Cache([900, 400], [300, 9], 2, 16, torch.bfloat16, seed=2)
    pages, batch, Q, out, _ = _attend(J, c, 8, max_q=2 ** 31 - 1)

    def call(num_seqs, total, max_q, max_pages):
        d = J.BatchDesc(num_seqs, total, max_q, max_pages, *(x.data_ptr() for x in (c.q_start, c.kv_len, c.table)))
        q = J._QUERIES.pack(Q.data_ptr(), 8 * D, D, 0, 0, out.data_ptr(), 0, 8, 1, SCALE)
        return J._lib.jolt_paged_attention(pages.handle, ctypes.addressof(d), q, None)

    before = J.jolt_launch_count()
    assert call(2, 309, 309, 1 << 27) == 9              # a table of 2^31 tokens
    assert call(1 << 30, 309, 309, 57) == 9             # 2^31 items
    assert call(2, 1 << 23, 1 << 23, 1 << 22) == 9      # 2^17 blocks of rows by 2^19 tiles of keys
    assert call(2, 1 << 28, 1, 57) == 9                 # 2^31 query rows
    assert J.jolt_launch_count() == before


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv,chunks,heads,g", [
    ([300, 40, 2], [2, 3, 2], 2, 2),         # up to 8 rows, clusters
    ([30000, 40], [2, 2], 2, 4),             # in many shares
    ([30000, 77], [4, 3], 2, 4),             # up to 16
    ([300, 5], [7, 5], 2, 4),                # up to 32, clusters
    ([30000, 140], [7, 8], 2, 4),
    ([30000, 40], [30, 40], 2, 4),           # chunks of half a block and less, in many shares
    ([30000, 140], [100, 140], 2, 4),        # whole blocks, in many shares
    ([100, 300], [130, 300], 3, 1),          # more tokens than the cache holds
    ([256] * 80, [256] * 80, 2, 2),          # many more blocks than CTAs
])
def test_values_that_are_no_numbers_where_they_are_not_seen(J, dtype, kv, chunks, heads, g):
    """Tokens of a chunk whose keys and values are no numbers (a padded chunk, say): the rows before them are
    as they should be, and the rows that see such a value show it, in its feature alone: as no finite number, which
    of them is open (a weight enters the product as a rounded part and a remainder that may be 0 or negative,
    and inf * hi + inf * lo is then inf + NaN or inf - inf)."""
    import torch
    c = Cache(kv, chunks, heads, 16, _t(dtype), seed=6)
    Q = c.randn(c.total, heads * g, D, scale=2.0)
    pages, batch = c.handles(J)
    seen = torch.zeros((c.total, heads * g, D), device="cuda")         # what every output is to show
    K0, V0 = c.K.clone(), c.V.clone()
    for s, (T, n) in enumerate(zip(kv, chunks)):
        for back, h, f, x in ((0, 0, 0, math.nan), (1, heads - 1, 50, math.inf), (n // 2, 0, 127, -math.inf)):
            t = T - 1 - back                                            # seen by the chunk's last 1 + back tokens
            c.V[c.table[s, t // 16].long(), h, t % 16, f] = x
            V0[c.table[s, t // 16].long(), h, t % 16, f] = 0.0
            seen[c.starts[s + 1] - 1 - back:c.starts[s + 1], h * g:(h + 1) * g, f] += x
    out = torch.zeros((c.total, heads * g, D), dtype=c.dtype, device="cuda")
    L = torch.zeros((c.total, heads * g), device="cuda")
    J.jolt_paged_attention(pages, batch, Q, out, SCALE, lse=L)
    J.jolt_pages_status(pages)
    bad = seen != 0                                                     # (a NaN is unequal to 0)
    assert not torch.isfinite(out[bad].float()).any()
    clean = Cache(kv, chunks, heads, 16, _t(dtype), seed=6)
    clean.V = V0
    ref = attention_ref(clean, Q, SCALE, True)[0]
    out[bad] = ref[bad].to(c.dtype)
    check_attention(clean, Q, out, L, SCALE, True)

    # the chunk's last token, keys too: it alone is no number, and so is its row
    c.V.copy_(V0)
    for s, T in enumerate(kv):
        c.K[c.table[s, (T - 1) // 16].long(), :, (T - 1) % 16] = math.nan
        c.V[c.table[s, (T - 1) // 16].long(), :, (T - 1) % 16] = math.inf
    J.jolt_paged_attention(pages, batch, Q, out, SCALE, lse=L)
    J.jolt_pages_status(pages)
    last = torch.tensor(c.starts[1:], device="cuda") - 1
    assert torch.isnan(out[last].float()).all() and torch.isnan(L[last]).all()
    ro, rl = attention_ref(clean, Q, SCALE, True)[:2]
    out[last], L[last] = ro[last].to(c.dtype), rl[last].float()
    check_attention(clean, Q, out, L, SCALE, True)


@pytest.mark.parametrize("hq,hk", [(65, 0), (60, 5), (40, 40), (200, 3)])
@pytest.mark.parametrize("inter", [False, True])
def test_tokens_of_many_rows(J, hq, hk, inter):
    """Tokens of one row more than a CTA takes at once, and of several times as many."""
    test_norm_rope(J, "bf16", 5, hq, hk, True, 128, inter, 4000)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("seqs,heads,g,n,kv", [
    (2, 8, 4, 4, 400), (2, 8, 4, 4, 7000), (3, 8, 4, 3, 7900), (4, 8, 4, 4, 8000), (4, 8, 4, 4, 9000), (9, 8, 4, 4, 300),
    (1, 8, 5, 4, 300), (2, 8, 4, 8, 500), (3, 8, 4, 8, 500), (4, 8, 4, 7, 510), (4, 8, 4, 7, 600), (5, 8, 4, 6, 200),
])
def test_nine_to_thirty_two_rows(J, dtype, seqs, heads, g, n, kv):
    """Either side of the sizes where the kernel for few rows gives way to the other one."""
    c = Cache([max(n, kv - 7 * s) for s in range(seqs)], [n - s % 2 for s in range(seqs)], heads, 16, _t(dtype), seed=n, pad=2)
    _attend(J, c, heads * g, max_q=n)
    _attend(J, c, heads * g, max_q=n, prefix=True, causal=False)
