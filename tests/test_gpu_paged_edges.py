"""Where the growing cache's operators can go wrong without a shape that looks odd: bad offsets that fall, reports made
while another stream works, weights far below the largest, prefixes that hold no number, precision. Bounds are derived
beside the tests, from paged_common's where nothing is said."""
import math

import pytest

from paged_common import D, Cache, check_attention, half_step

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


def _reported(J, pages, **kw):
    """What jolt_pages_status says, or nothing."""
    try:
        J.jolt_pages_status(pages, **kw)
    except J.JoltError as e:
        assert e.status == 1
        return str(e)
    return ""


def test_append_of_tokens_that_two_sequences_claim(J):
    """Offsets that fall make the sequences around them overlap. Each token is then appended for one of them, the
    last, at the place that this one has for it: never by one's table and another's position, whose table entry may
    lie behind the sequence's pages and name a page of someone else."""
    import torch
    S, n, page = 301, 40, 16
    kv = [n + 16 * (s % 7) for s in range(S)]
    own = [(t + page - 1) // page for t in kv]
    cols = max(own)
    table = torch.zeros((S, cols), dtype=torch.int32)
    at = 0
    for s in range(S):
        table[s, :own[s]] = torch.arange(at, at + own[s])
        table[s, own[s]:] = sum(own)                      # not among the sequence's pages: a page of someone else
        at += own[s]
    K = torch.zeros((at + 1, 1, page, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    pages = J.jolt_pages_create(K, V)
    starts = [0 if s % 2 == 0 else n for s in range(S + 1)]       # 0 40 0 40 ...: every other sequence falls
    batch = J.jolt_batch(torch.tensor(starts, dtype=torch.int32, device="cuda"),
                         torch.tensor(kv, dtype=torch.int32, device="cuda"), table.cuda(), n, n)
    last = S - 1
    assert starts[last] == 0 and starts[S] == n
    pos = torch.arange(kv[last] - n, kv[last])
    want_p, want_r = table[last][pos // page].long().cuda(), (pos % page).cuda()
    g = torch.Generator(device="cuda").manual_seed(1)
    for _ in range(200):
        x = torch.randn((n, 2, D), generator=g, device="cuda").to(torch.bfloat16)
        K.zero_(), V.zero_()
        J.jolt_paged_append(pages, batch, x[:, :1], x[:, 1:])
        _reported(J, pages)
        for X, new in ((K, x[:, 0]), (V, x[:, 1])):
            assert torch.equal(X[want_p, 0, want_r], new)
            X[want_p, 0, want_r] = 0
            assert not X.any(), X.flatten(1).any(1).nonzero()[:4].tolist()


@pytest.mark.parametrize("starts,kv,total", [
    ([0, 3, 1, 4], [9, 9, 9], 4),            # an offset that falls between two tokens
    ([0, 4, 9], [9, 9], 4),                  # a sequence wholly behind the batch's rows
    ([0, 4, -3], [9, 9], 4),
    ([0, 4, 4], [9, -5], 4),                 # a length below zero, or beyond the table, of a sequence without tokens
    ([0, 4, 4], [9, 17], 4),
])
def test_append_reports_what_attention_reports(J, starts, kv, total):
    import torch
    K = torch.zeros((8, 2, 16, D), dtype=torch.bfloat16, device="cuda")
    V = torch.zeros_like(K)
    pages = J.jolt_pages_create(K, V)
    i32 = dict(dtype=torch.int32, device="cuda")
    batch = J.jolt_batch(torch.tensor(starts, **i32), torch.tensor(kv, **i32), torch.arange(len(kv), **i32)[:, None].contiguous(),
                         total, total)
    x = torch.ones((total, 2, D), dtype=torch.bfloat16, device="cuda")
    J.jolt_paged_append(pages, batch, x, x)
    assert "q_start or kv_len" in _reported(J, pages)
    assert not _reported(J, pages)
    J.jolt_paged_attention(pages, batch, x, torch.empty_like(x), SCALE)
    assert "q_start or kv_len" in _reported(J, pages)


def test_no_report_is_lost_to_another_stream(J):
    """A batch is found wrong on one stream while the reports are fetched on another: each is seen once."""
    import torch
    c = Cache([40], [1], 1, 16, torch.bfloat16, poison=False)
    pages, batch = c.handles(J)
    c.kv_len.fill_(-1)
    x = c.randn(1, 1, D)
    work, ask = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    lost = 0
    for i in range(4000):
        with torch.cuda.stream(work):
            torch.cuda._sleep(500 * (i % 64))            # up to 16 us: the report falls anywhere into the fetching
            J.jolt_paged_append(pages, batch, x, x)
        done = work.record_event()
        seen = 0
        while not done.query():
            seen += bool(_reported(J, pages, cuda_stream=ask))
        seen += bool(_reported(J, pages, cuda_stream=ask))
        lost += seen == 0
        assert seen <= 1
    assert lost == 0


def test_a_report_names_all_that_was_found(J):
    import torch
    c = Cache([40, 40], [1, 1], 1, 16, torch.bfloat16, poison=False)
    pages, batch = c.handles(J)
    c.kv_len[0] = -1
    c.table[1] = -3
    x = c.randn(2, 1, D)
    J.jolt_paged_append(pages, batch, x, x)
    said = _reported(J, pages)
    assert "q_start or kv_len" in said and "page table" in said


@pytest.mark.parametrize("kv,chunks", [([0, 40], [1, 1]), ([0, 40], [5, 5]), ([0, 40], [40, 40]), ([0, 400], [300, 300]),
                                       ([0, 9000], [1, 1])])
def test_a_prefix_that_is_no_number_shows(J, kv, chunks):
    """A log-sum-exp of a prefix that is no number makes its row none, also a row that has no keys."""
    import torch
    c = Cache(kv, chunks, 2, 16, torch.bfloat16, seed=3)
    Q, out = c.randn(c.total, 8, D), torch.zeros((c.total, 8, D), dtype=c.dtype, device="cuda")
    L = torch.zeros((c.total, 8), device="cuda")
    po, pl = c.randn(c.total, 8, D, dtype=torch.float32), c.randn(c.total, 8, dtype=torch.float32)
    rows = [0, c.starts[1] - 1, c.starts[1], c.total - 1]
    pl[rows, 3] = math.nan
    pages, batch = c.handles(J)
    J.jolt_paged_attention(pages, batch, Q, out, SCALE, lse=L, prefix_out=po, prefix_lse=pl)
    J.jolt_pages_status(pages)
    assert torch.isnan(out[rows, 3].float()).all() and torch.isnan(L[rows, 3]).all()
    pl[rows, 3] = 0.5
    good, G = torch.zeros_like(out), torch.zeros_like(L)
    J.jolt_paged_attention(pages, batch, Q, good, SCALE, lse=G, prefix_out=po, prefix_lse=pl)
    out[rows, 3], L[rows, 3] = good[rows, 3], G[rows, 3]
    assert torch.equal(out, good) and torch.equal(L, G)


@pytest.mark.parametrize("chunks", [[1, 1], [40, 9]])
def test_a_scale_that_is_no_finite_number_is_refused(J, chunks):
    import torch
    c = Cache([100, 60], chunks, 2, 16, torch.bfloat16, seed=1)
    Q = c.randn(c.total, 8, D)
    pages, batch = c.handles(J)
    before = J.jolt_launch_count()
    for scale in (math.nan, math.inf, -math.inf):
        with pytest.raises(J.JoltError) as e:
            J.jolt_paged_attention(pages, batch, Q, torch.empty_like(Q), scale)
        assert e.value.status == 1 and "scale" in str(e.value)
    assert J.jolt_launch_count() == before


def _stream(J, tokens, heads):
    import synth
    from gpu_common import gpu_encode
    cfg = synth.config(1, layers=2, tokens=tokens, heads=heads, seed=1709, groups=2)
    K, V = synth.gen_cache_numpy(cfg)
    return gpu_encode(cfg, K, V, synth.bf16_bytes(cfg) // 2, "sketch")[1]


def test_attention_over_a_stream_of_many_queries(J):
    """As many queries as a grid's dimension does not hold groups of, in bounded scratch; each row as in a call of few."""
    import torch
    st = _stream(J, 300, 1)
    n, hq = 65536 + 77, 4
    g = torch.Generator(device="cuda").manual_seed(4)
    Q = torch.randn((n, hq, D), generator=g, device="cuda").to(torch.bfloat16)
    out, L = torch.full((n, hq, D), math.nan, device="cuda"), torch.full((n, hq), math.nan, device="cuda")
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    J.jolt_attention_lse(st, 1, Q, out, L, SCALE)
    torch.cuda.synchronize()
    assert free - torch.cuda.mem_get_info()[0] <= 400 << 20
    for at in (0, 5, 1023, 30000, n - 9):
        o, l = torch.empty((9, hq, D), device="cuda"), torch.empty((9, hq), device="cuda")
        J.jolt_attention_lse(st, 1, Q[at:at + 9], o, l, SCALE)
        assert torch.equal(o, out[at:at + 9]) and torch.equal(l, L[at:at + 9])
    assert torch.isfinite(out).all() and torch.isfinite(L).all()


def test_attention_over_a_stream_beyond_its_grid_is_refused(J):
    """All layers at once, more groups of queries than the grid's third dimension holds: refused before any launch."""
    import torch
    st = _stream(J, 300, 1)
    Q = torch.zeros((2, 4, 32768, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty(Q.shape, device="cuda")
    before = J.jolt_launch_count()
    with pytest.raises(J.JoltError) as e:
        J.jolt_attention(st, Q, out, SCALE)
    assert e.value.status == 9 and J.jolt_launch_count() == before


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("below", [16, 18, 20])
@pytest.mark.parametrize("seqs,n,g", [(2, 1, 4), (600, 1, 4), (600, 3, 4), (300, 5, 4), (300, 100, 1), (300, 200, 1)])
def test_many_keys_far_below_one(J, dtype, below, seqs, n, g):
    """One key whose value is 0, and 32767 others `below` lower in the exponent: they make the output, each with a
    weight that 16 bits would not hold beside 1.

    The bound: a score is 8 below / 8 in one product, exact, but for its scale in units of log 2 (2 roundings of
    2^-24 of a number up to 29, each moving a weight by 2 ln 2 times as much: 2^-17); the weights' and the output's
    rounding (2 half steps), sums in 32 bits over 2^15 keys in blocks (2^-15 with each of 2^11 accumulations off by a
    last place); and what is below the type's smallest numbers, half of fp16's, 2^-25, beside a largest
    weight of 2^9 at least: 2^-34 a key."""
    import torch
    t, kv, page = _t(dtype), 32768, 64
    K = torch.zeros((kv // page, 1, page, D), dtype=t, device="cuda")
    V = torch.zeros_like(K)
    v = torch.linspace(-1, 1, D, device="cuda").to(t)
    V[:] = v
    V[0, 0, 0] = 0
    K[0, 0, 0, 5] = below
    pages = J.jolt_pages_create(K, V)
    table = torch.arange(kv // page, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()   # all share them
    Q = torch.zeros((seqs * n, g, D), dtype=t, device="cuda")
    Q[..., 5] = 8
    out = torch.full_like(Q, math.nan)
    L = torch.full((seqs * n, g), math.nan, device="cuda")
    batch = J.jolt_batch(n * torch.arange(seqs + 1, dtype=torch.int32, device="cuda"),
                         torch.full((seqs,), kv, dtype=torch.int32, device="cuda"), table, seqs * n, n)
    J.jolt_paged_attention(pages, batch, Q, out, 0.125, lse=L)
    J.jolt_pages_status(pages)
    many = (kv - n + torch.arange(n, device="cuda")).double().repeat(seqs)[:, None, None]     # keys but the first
    w = many * math.exp(-below)
    ref = w / (1 + w) * v.double()
    h = half_step(t)
    tol = (2 * h + 2.0 ** -15 + 2.0 ** -17) * ref.abs() + torch.finfo(t).tiny * h
    if t == torch.float16:
        tol += 2.0 ** -34 * kv * v.double().abs()
    err = (out.double() - ref).abs()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()))
    ref_l = torch.log(math.exp(below) + many[..., 0])
    assert ((L.double() - ref_l).abs() <= 2.0 ** -15 + 2.0 ** -22 * below).all(), float((L.double() - ref_l).abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("kv,chunks,heads,g", [
    ([300, 77, 200], [1, 1, 1], 2, 4),           # up to 8 rows, clusters
    ([300, 77, 200] * 20, [2, 1, 2] * 20, 2, 4),  # in shares
    ([300, 77, 200], [3, 4, 2], 2, 4),           # up to 16 rows
    ([300, 77, 200], [5, 8, 6], 1, 4),           # up to 32
    ([300, 77, 200] * 20, [3, 4, 2] * 20, 2, 4),  # the same of many sequences
    ([300, 77, 200] * 20, [5, 8, 6] * 20, 2, 4),
    ([300, 150, 200], [100, 128, 127], 2, 1),    # up to 128
    ([300, 150, 200] * 30, [100, 128, 33] * 30, 2, 1),
])
def test_up_to_128_rows_round_the_output_alone(J, dtype, kv, chunks, heads, g):
    """Up to 128 rows that read one KV head of a sequence: their weights are not rounded to the type, whatever else
    is in the batch, so that the output's rounding is all that is left.

    Queries and keys are small whole numbers and the scale is a power of two, so scores are exact. What remains, of
    A = sum_j w_j |v_j|: their scale in units of log 2 (2 roundings of 2^-24 of up to 64, times 2 ln 2: 2^-16), the
    weights' remainder, rounded to the type (h^2), and the sums: up to 2 x 300 / 16 accumulations, off by a last place
    each (2^-17). Without the remainder it would be h, 2^-8 in bf16."""
    import torch
    t = _t(dtype)
    c = Cache(kv, chunks, heads, 16, t, seed=len(kv))
    c.K.copy_(torch.where(torch.isnan(c.K), c.K, torch.randint(-2, 3, c.K.shape, generator=c.g, device="cuda").to(t)))
    Q = torch.randint(-2, 3, (c.total, heads * g, D), generator=c.g, device="cuda").to(t)
    out, L = torch.full_like(Q, math.nan), torch.full((c.total, heads * g), math.nan, device="cuda")
    pages, batch = c.handles(J)
    J.jolt_paged_attention(pages, batch, Q, out, 0.125, lse=L)
    J.jolt_pages_status(pages)
    check_attention(c, Q, out, L, 0.125, True)
    h = half_step(t)
    for s in range(len(kv)):
        n, r = c.n[s], slice(c.starts[s], c.starts[s + 1])
        for k in range(heads):
            K, V = c.rows(s, k, c.K).double(), c.rows(s, k, c.V).double()
            x = Q[r, k * g:k * g + g].double()
            z = (x @ K.T * 0.125).masked_fill(torch.arange(kv[s], device="cuda") > (kv[s] - n + torch.arange(n, device="cuda"))[:, None, None],
                                              -math.inf)
            assert z[z > -math.inf].abs().max() * math.log2(math.e) < 64
            w = torch.softmax(z, -1)
            ref, A = w @ V, w @ V.abs()
            tol = h * ref.abs() + (1 + h) * (h * h + 2.0 ** -16 + 2.0 ** -17) * A + torch.finfo(t).tiny
            err = (out[r, k * g:k * g + g].double() - ref).abs()
            assert (err <= tol).all(), (s, k, float((err / tol).max()))


@pytest.mark.parametrize("n", [1, 4])
def test_one_long_sequence_among_few(J, n):
    """Four sequences of eight KV heads, one of them long: its keys are divided over the whole GPU and their parts combined
    by a second launch, where a cluster an item would leave it to an eighth of the CTAs; small tables stay with clusters."""
    import torch
    for long, launches in ((16384 - n, 2), (8000, 2), (4000, 1)):
        if n > 1 and long > 8192:
            continue
        c = Cache([long, 100, 7, 60], [n] * 4, 8, 16, torch.bfloat16, seed=n)
        Q = c.randn(c.total, 32, D)
        out, L = torch.full_like(Q, math.nan), torch.full((c.total, 32), math.nan, device="cuda")
        pages, batch = c.handles(J)
        before = J.jolt_launch_count()
        J.jolt_paged_attention(pages, batch, Q, out, SCALE, lse=L)
        assert J.jolt_launch_count() - before == launches
        J.jolt_pages_status(pages)
        check_attention(c, Q, out, L, SCALE, True)


def test_a_stream_from_the_host_knows_its_layers(J):
    import torch
    st = _stream(J, 300, 1)
    back = J.jolt_stream_from_host(J.jolt_stream_to_host(st))
    Q = torch.randn((2, 4, 3, D), device="cuda").to(torch.bfloat16)
    a, b = torch.zeros(Q.shape, device="cuda"), torch.ones(Q.shape, device="cuda")
    J.jolt_attention(st, Q, a, SCALE)
    J.jolt_attention(back, Q, b, SCALE)
    assert torch.equal(a, b)
    for s in (st, back):
        with pytest.raises(ValueError):
            J.jolt_attention(s, Q[:1], a[:1], SCALE)


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("scale", [0.0025, 0.0884, 0.3536, -0.0884])
@pytest.mark.parametrize("seqs,n,g", [(2, 1, 4), (300, 1, 4), (2, 3, 4), (40, 5, 4), (2, 200, 1), (160, 200, 1)])
def test_scores_of_millions(J, dtype, scale, seqs, n, g):
    """Scores whose last places are whole units of the exponent, rising by less than a weight's range from tile to tile:
    no weight may leave the type's range for it, so each output stays between the values and near those of the
    largest scores: a score is exact, 2^24 to 2^26 in units of log 2, and its rounding moves a weight by 2^4 at most, so
    keys 24 and more below the row's largest have less than 900 2^-16 of it together."""
    import torch
    t, kv, page = _t(dtype), 900, 64
    big = 1024.0                                   # 127 products of 2^20, exact
    K = torch.full((15, 1, page, D), big, device="cuda").to(t)
    j = torch.arange(15 * page, device="cuda").reshape(15, page)
    rise = (j // 32).float() if scale > 0 else (30 - j // 32).float()
    K[:, 0, :, 127] = (8 * rise if dtype == "f16" else rise).to(t)      # bf16 holds whole numbers up to 256
    V = torch.randn((15, 1, page, D), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(t)
    Q = torch.full((seqs * n, g, D), big, device="cuda").to(t)
    Q[..., 127] = 8 if dtype == "bf16" else 1
    pages = J.jolt_pages_create(K, V)
    table = torch.arange(15, dtype=torch.int32, device="cuda").expand(seqs, -1).contiguous()
    batch = J.jolt_batch(n * torch.arange(seqs + 1, dtype=torch.int32, device="cuda"),
                         torch.full((seqs,), kv, dtype=torch.int32, device="cuda"), table, seqs * n, n)
    out, L = torch.full_like(Q, math.nan), torch.full((seqs * n, g), math.nan, device="cuda")
    J.jolt_paged_attention(pages, batch, Q, out, scale, lse=L)
    J.jolt_pages_status(pages)
    assert torch.isfinite(out.float()).all() and torch.isfinite(L).all()
    v = V.reshape(-1, D)[:kv].double()
    z = (K.reshape(-1, D)[:kv].double() @ Q[0, 0].double()) * scale * math.log2(math.e)
    for i in {0, n - 1, n // 2}:
        see = kv - n + i + 1
        near = z[:see] > z[:see].max() - 24
        lo, hi = v[:see][near].amin(0), v[:see][near].amax(0)
        slack = half_step(t) * 4 + 2.0 ** -5
        o = out.reshape(seqs, n, g, D)[:, i].double()
        assert (o >= lo - slack).all() and (o <= hi + slack).all(), (i, float((lo - o).max()), float((o - hi).max()))
