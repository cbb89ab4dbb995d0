"""Measured cases of the operators of the growing cache: the norm and rotation of queries and keys,
the append to a paged cache, and the attention of new tokens over it (jolt_qk_norm_rope,
jolt_paged_append, jolt_paged_attention).

`run(state)` computes a case with elementary torch operations in 32 bits (angles in 64) when `own`
is false, and with the library's entry points when it is true. Sizes come from the workloads of
synth/kv.py (8 KV heads as in Mistral-7B with 32 query heads, 40 heads as in LLaMA-2-13B; contexts
of 1024, 4096, 8192 and 32768 tokens) or are generic.
"""
import math

import numpy as np
import torch

own = False
D = 128
EPS = 1e-6


def _attn(name, **kw):
    c = dict(name=name, op="attention", dtype="bf16", seqs=1, q_heads=32, heads=8, page=16, q_min=1, q_max=1,
             kv_min=1024, kv_max=1024, causal=True, prefix=False, idle=0, pad=0)
    c.update(kw)
    return c


def listed():
    return [
        # one sequence generating over a 1024-token cache: the latency of the smallest call
        _attn("decode_b1_t1024"),
        # a serving batch of sequences of very different lengths, two graph slots unused
        _attn("decode_b64_ragged_t8192", seqs=64, kv_min=1, kv_max=8192, idle=2),
        # one long document: few rows, so the key axis has to be split over the whole GPU
        _attn("decode_b1_t131072", kv_min=131072, kv_max=131072, page=64),
        # multi-head attention (one query row a head) in fp16
        _attn("decode_f16_mha_b16_t4096", seqs=16, q_heads=40, heads=40, kv_min=4096, kv_max=4096, dtype="f16", page=32),
        # drafted tokens checked in one call, behind a prefix that is attended elsewhere
        _attn("draft_b16_n5_prefix", seqs=16, q_min=2, q_max=5, kv_min=512, kv_max=4096, prefix=True, page=128),
        # chunked prefill and generation in one batch, padded rows behind the last sequence
        _attn("mixed_b24_n512_t8192", seqs=24, q_min=1, q_max=512, kv_min=513, kv_max=8192, page=64, pad=37),
        # a whole prompt
        _attn("prefill_t8192", q_min=8192, q_max=8192, kv_min=8192, kv_max=8192, page=64),
        # one chunk of a long prompt
        _attn("chunk_n2048_t32768", q_min=2048, q_max=2048, kv_min=32768, kv_max=32768, page=128),
        # a generation step and a prompt written to the pages, keys rotated (and normed) on the way
        dict(name="append_b64", op="append", dtype="bf16", seqs=64, heads=8, page=16, q_min=1, q_max=1, kv_min=1,
             kv_max=256, norm=False, rope=128, interleaved=False, start=32768),
        dict(name="append_t8192_norm", op="append", dtype="bf16", seqs=2, heads=8, page=64, q_min=8191, q_max=8191,
             kv_min=8191, kv_max=8200, norm=True, rope=128, interleaved=False, start=0),
        # queries and keys of a generation step and of a prompt
        dict(name="norm_rope_n64", op="norm_rope", dtype="bf16", tokens=64, q_heads=32, heads=8, norm=True, rope=128,
             interleaved=False, start=131000),
        dict(name="norm_rope_f16_n16384", op="norm_rope", dtype="f16", tokens=16384, q_heads=40, heads=40, norm=True,
             rope=128, interleaved=False, start=0),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "append", "norm_rope"])
    dtype = rng.choice(["bf16", "bf16", "f16"])
    heads = rng.choice([1, 2, 4, 5, 8, 8, 10, 16, 40])
    g = rng.choice([1, 2, 3, 4, 4, 5, 7, 8, 16])
    while heads * g > 64:
        g = max(1, g // 2)
    page = rng.choice([16, 16, 32, 48, 64, 128, 256])
    if op == "norm_rope":
        tokens = min(_log(rng, 1, 16384), 16384 * 80 // (heads * (g + 1)))
        return dict(op=op, dtype=dtype, tokens=tokens, q_heads=heads * g, heads=heads, norm=rng.random() < 0.7,
                    rope=rng.choice([32, 64, 96, 128, 128]), interleaved=rng.random() < 0.4, start=_log(rng, 1, 500000))
    if op == "append":
        q_max = _log(rng, 1, 4096)
        seqs = max(1, min(_log(rng, 1, 128), 16384 * 8 // (q_max * heads)))
        return dict(op=op, dtype=dtype, seqs=seqs, heads=heads, page=page, q_min=rng.choice([1, q_max]), q_max=q_max,
                    kv_min=q_max, kv_max=q_max + _log(rng, 1, 512), norm=rng.random() < 0.5,
                    rope=rng.choice([64, 128, 128]), interleaved=rng.random() < 0.4, start=_log(rng, 1, 500000))
    q_max = rng.choice([1, 1, _log(rng, 2, 16), _log(rng, 16, 2048)])
    kv_max = max(q_max, _log(rng, 1, 65536))
    seqs = _log(rng, 1, 128)
    # no dearer than the largest listed cases: pairs of the plain form's padded scores, padded keys
    while seqs > 1 and (seqs * q_max * kv_max * heads * g > 2 ** 30 or seqs * kv_max * heads > 2 ** 22):
        seqs = max(1, seqs // 2)
    while q_max > 1 and seqs * q_max * kv_max * heads * g > 2 ** 30:
        q_max = max(1, q_max // 2)
    return dict(op=op, dtype=dtype, seqs=seqs, q_heads=heads * g, heads=heads, page=page, q_min=rng.choice([1, q_max]),
                q_max=q_max, kv_min=rng.choice([q_max, kv_max]), kv_max=kv_max, causal=rng.random() < 0.8,
                prefix=rng.random() < 0.3, idle=rng.choice([0, 0, 1]) if seqs > 2 else 0, pad=rng.choice([0, 0, 19]))


def _lengths(case):
    """Chunk and cache lengths of each sequence, spread over the case's ranges: the same for every
    seed, so that a case is the same work."""
    S = case["seqs"]
    r = np.random.default_rng(S * 7919 + case["kv_max"])
    n = r.integers(case["q_min"], case["q_max"] + 1, S)
    kv = r.integers(case["kv_min"], case["kv_max"] + 1, S)
    n[r.integers(0, S)] = case["q_max"]
    kv[r.integers(0, S)] = case["kv_max"]
    kv = np.maximum(kv, n)
    if case.get("idle"):
        kv[S - case["idle"]:] = 0          # slots of a captured batch that hold no sequence
        n[S - case["idle"]:] = 1
    return n, kv


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float16


def _freqs(case):
    r = case["rope"]
    return (1.0e6 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _dtype(case)

    def randn(*shape, scale=1.0, dtype=t):
        return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * scale).to(dtype)

    st = {"case": case, "op": case["op"]}
    if case["op"] == "norm_rope":
        N, Hq, H = case["tokens"], case["q_heads"], case["heads"]
        qkv = randn(N, Hq + 2 * H, D, scale=1.5)             # the fused projection's output
        st["Q"], st["K"] = qkv[:, :Hq], qkv[:, Hq:Hq + H]
        st["positions"] = (case["start"] + torch.randperm(N, generator=g, device="cuda")).to(torch.int32)
        st["inv_freq"] = _freqs(case)
        st["qw"] = (1 + randn(D, scale=0.2, dtype=torch.float32)).to(t) if case["norm"] else None
        st["kw"] = (1 + randn(D, scale=0.2, dtype=torch.float32)).to(t) if case["norm"] else None
        st["Q_out"] = torch.empty((N, Hq, D), dtype=t, device="cuda")
        st["K_out"] = torch.empty((N, H, D), dtype=t, device="cuda")
        return st
    n, kv = _lengths(case)
    S, H, P = case["seqs"], case["heads"], case["page"]
    need = (kv + P - 1) // P
    total = int(need.sum())
    pool = total + 3
    st["K_pages"] = randn(pool, H, P, D)
    st["V_pages"] = randn(pool, H, P, D)
    perm = torch.randperm(pool, generator=g, device="cuda").cpu().numpy()[:total]
    table = np.full((S, max(1, int(need.max()))), -1, dtype=np.int32)   # entries behind a sequence's pages hold no page
    at = 0
    for s in range(S):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    starts = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    N = int(starts[-1]) + case.get("pad", 0)
    st["q_start"] = torch.from_numpy(starts).cuda()
    st["kv_len"] = torch.from_numpy(kv.astype(np.int32)).cuda()
    st["table"] = torch.from_numpy(table).cuda()
    st["total_q"], st["max_q"] = N, int(n.max())
    if case["op"] == "append":
        qkv = randn(N, 3 * H, D, scale=1.5)
        st["K"], st["V"] = qkv[:, H:2 * H], qkv[:, 2 * H:]
        st["positions"] = (case["start"] + torch.arange(N, device="cuda")).to(torch.int32)
        st["inv_freq"] = _freqs(case)
        st["kw"] = (1 + randn(D, scale=0.2, dtype=torch.float32)).to(t) if case["norm"] else None
    else:
        Hq = case["q_heads"]
        st["Q"] = randn(N, Hq, D, scale=2.0)
        st["scale"] = 1.0 / math.sqrt(D)
        st["causal"] = case["causal"]
        if case["prefix"]:
            st["prefix_out"] = randn(N, Hq, D, scale=0.3, dtype=torch.float32)
            st["prefix_lse"] = randn(N, Hq, dtype=torch.float32) + math.log(max(1, case["kv_max"]))
        st["out"] = torch.zeros((N, Hq, D), dtype=t, device="cuda")
        st["lse"] = torch.zeros((N, Hq), dtype=torch.float32, device="cuda")
    if own:
        from tensor_decomposition_b200 import jolt as J
        st["pages"] = J.jolt_pages_create(st["K_pages"], st["V_pages"])
        st["batch"] = J.jolt_batch(st["q_start"], st["kv_len"], st["table"], st["total_q"], st["max_q"])
    return st


# ------------------------------------------------------------------ plain forms
def _norm(x, w):
    return x if w is None else x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(x.dtype)


def _rotate(x, positions, inv_freq, interleaved):
    """x [tokens][heads][128], the first 2 len(inv_freq) features of each row rotated."""
    h = inv_freq.numel()
    a = positions.double()[:, None, None] * inv_freq.double()
    c, s = torch.cos(a).to(x.dtype), torch.sin(a).to(x.dtype)
    r, rest = x[..., :2 * h], x[..., 2 * h:]
    if interleaved:
        u, v = r[..., 0::2], r[..., 1::2]
        r = torch.stack((u * c - v * s, v * c + u * s), dim=-1).flatten(-2)
    else:
        u, v = r[..., :h], r[..., h:]
        r = torch.cat((u * c - v * s, v * c + u * s), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _slots(st, page):
    """(sequence, index in its chunk) of every token of the batch, and the page and row it is kept in."""
    q0 = st["q_start"].long()
    i = torch.arange(st["K"].shape[0], device="cuda")
    s = torch.searchsorted(q0, i, right=True) - 1
    pos = st["kv_len"].long()[s] - (q0[s + 1] - i)
    return st["table"].long()[s, pos // page], pos % page


def _append(st, K, V):
    page, row = _slots(st, st["case"]["page"])
    st["K_pages"][page, :, row] = K.to(st["K_pages"].dtype)
    st["V_pages"][page, :, row] = V
    return {"K_pages": st["K_pages"], "V_pages": st["V_pages"]}


def _attention(st):
    Q, t = st["Q"], st["Q"].dtype
    table, kv_len, q0 = st["table"].long().clamp(min=0), st["kv_len"].long(), st["q_start"].long()
    S, H, Hq = table.shape[0], st["K_pages"].shape[1], Q.shape[1]
    g, mq = Hq // H, st["max_q"]
    K = st["K_pages"][table].float().transpose(1, 2).reshape(S, H, -1, D)
    V = st["V_pages"][table].float().transpose(1, 2).reshape(S, H, -1, D)
    T = K.shape[2]
    n = q0[1:] - q0[:-1]
    i = torch.arange(mq, device="cuda")
    rows = q0[:-1, None] + i
    real = i < n[:, None]                                                     # [S][mq]
    q = Q[rows.clamp(max=Q.shape[0] - 1)].float().reshape(S, mq, H, g, D).permute(0, 2, 1, 3, 4)
    s = torch.matmul(q.reshape(S, H, mq * g, D), K.transpose(2, 3)).reshape(S, H, mq, g, T) * st["scale"]
    limit = (kv_len - n)[:, None] + i if st["causal"] else (kv_len - 1)[:, None].expand(S, mq)
    j = torch.arange(T, device="cuda")
    s.masked_fill_((j > limit[:, :, None])[:, None, :, None, :], -math.inf)
    m = s.amax(-1, keepdim=True)
    if "prefix_lse" in st:
        pad = rows.clamp(max=Q.shape[0] - 1)
        pl = st["prefix_lse"][pad].reshape(S, mq, H, g).permute(0, 2, 1, 3)[..., None]
        po = st["prefix_out"][pad].reshape(S, mq, H, g, D).permute(0, 2, 1, 3, 4)
        m = torch.maximum(m, pl)
    m = torch.where(m == -math.inf, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    V = torch.where((j < kv_len[:, None])[:, None, :, None], V, 0.0)
    o = torch.matmul(p.reshape(S, H, mq * g, T), V).reshape(S, H, mq, g, D)
    if "prefix_lse" in st:
        w = torch.exp(pl - m)
        l, o = l + w, o + w * po
    lse = (m + torch.log(l))[..., 0]
    o = o / torch.where(l == 0, 1.0, l)
    o = o.permute(0, 2, 1, 3, 4).reshape(S, mq, Hq, D)
    lse = lse.permute(0, 2, 1, 3).reshape(S, mq, Hq)
    st["out"][rows[real]] = o[real].to(t)
    st["lse"][rows[real]] = lse[real]
    return {"out": st["out"], "lse": st["lse"]}


def run(st):
    op, case = st["op"], st["case"]
    if own:
        from tensor_decomposition_b200 import jolt as J
        if op == "norm_rope":
            J.jolt_qk_norm_rope(st["Q"], st["Q_out"], st["K"], st["K_out"], positions=st["positions"],
                                inv_freq=st["inv_freq"], q_weight=st["qw"], k_weight=st["kw"], eps=EPS,
                                interleaved=case["interleaved"])
            return {"Q": st["Q_out"], "K": st["K_out"]}
        if op == "append":
            J.jolt_paged_append(st["pages"], st["batch"], st["K"], st["V"], positions=st["positions"],
                                inv_freq=st["inv_freq"], k_weight=st["kw"], eps=EPS, interleaved=case["interleaved"])
            return {"K_pages": st["K_pages"], "V_pages": st["V_pages"]}
        J.jolt_paged_attention(st["pages"], st["batch"], st["Q"], st["out"], st["scale"], causal=st["causal"],
                               lse=st["lse"], prefix_out=st.get("prefix_out"), prefix_lse=st.get("prefix_lse"))
        return {"out": st["out"], "lse": st["lse"]}
    if op == "norm_rope":
        t = st["Q"].dtype
        rot = (st["positions"], st["inv_freq"], case["interleaved"])
        st["Q_out"].copy_(_rotate(_norm(st["Q"].float(), st["qw"]), *rot).to(t))
        st["K_out"].copy_(_rotate(_norm(st["K"].float(), st["kw"]), *rot).to(t))
        return {"Q": st["Q_out"], "K": st["K_out"]}
    if op == "append":
        K = _rotate(_norm(st["K"].float(), st["kw"]), st["positions"], st["inv_freq"], case["interleaved"])
        return _append(st, K, st["V"])
    return _attention(st)


def work(case):
    row = 2 * D
    if case["op"] == "norm_rope":
        rows = case["tokens"] * (case["q_heads"] + case["heads"])
        return {"bytes": 2 * rows * row + 4 * case["tokens"], "flops": 8 * D * rows}
    n, kv = _lengths(case)
    H, N = case["heads"], int(n.sum())
    if case["op"] == "append":
        return {"bytes": 4 * N * H * row + 4 * N + 12 * len(n), "flops": 8 * D * N * H}
    Hq = case["q_heads"]
    pairs = 0
    for a, b in zip(n.tolist(), kv.tolist()):
        i = np.arange(a, dtype=np.int64)
        pairs += int(np.maximum(b - a + i + 1, 0).sum()) if case["causal"] else a * b
    io = 2 * N * Hq * row + 4 * N * Hq + (N * Hq * (4 * D + 4) if case["prefix"] else 0)
    return {"bytes": int(kv.sum()) * H * 2 * row + io, "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------ 64 bits, from the definition
def _exact_rows(X, w, positions, inv_freq, interleaved):
    X = X.double()
    if w is not None:
        X = X / torch.sqrt(torch.sum(X ** 2, -1, keepdim=True) / D + EPS) * w.double()
    Y = X.clone()
    r = 2 * inv_freq.numel()
    for i in range(r // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r // 2)
        ang = (positions.double() * inv_freq[i].double())[:, None]
        Y[..., a] = X[..., a] * torch.cos(ang) - X[..., b] * torch.sin(ang)
        Y[..., b] = X[..., a] * torch.sin(ang) + X[..., b] * torch.cos(ang)
    return Y


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        a = (st["positions"], st["inv_freq"], case["interleaved"])
        return {"Q": _exact_rows(st["Q"], st["qw"], *a), "K": _exact_rows(st["K"], st["kw"], *a)}
    q0, kv = st["q_start"].tolist(), st["kv_len"].tolist()
    P, H = case["page"], case["heads"]
    if case["op"] == "append":
        K = _exact_rows(st["K"], st["kw"], st["positions"], st["inv_freq"], case["interleaved"])
        Kp, Vp = st["K_pages"].double(), st["V_pages"].double()
        for s in range(case["seqs"]):
            n = q0[s + 1] - q0[s]
            pos = torch.arange(kv[s] - n, kv[s], device="cuda")
            page, row = st["table"][s].long()[pos // P], pos % P
            Kp[page, :, row] = K[q0[s]:q0[s + 1]]
            Vp[page, :, row] = st["V"][q0[s]:q0[s + 1]].double()
        return {"K_pages": Kp, "V_pages": Vp}
    g = case["q_heads"] // H
    out, lse = st["out"].double(), st["lse"].double()
    for s in range(case["seqs"]):
        n, T = q0[s + 1] - q0[s], kv[s]
        ids = st["table"][s, :(T + P - 1) // P].long()
        for h in range(H):
            K = st["K_pages"][ids, h].reshape(-1, D)[:T].double()
            V = st["V_pages"][ids, h].reshape(-1, D)[:T].double()
            for r0 in range(0, n, 4096):                                       # rows a bounded share at a time
                rows = slice(q0[s] + r0, q0[s] + min(n, r0 + 4096))
                for q in range(h * g, h * g + g):
                    z = st["Q"][rows, q].double() @ K.T * st["scale"]
                    if case["causal"]:
                        last = T - n + r0 + torch.arange(z.shape[0], device="cuda")
                        z[torch.arange(T, device="cuda")[None] > last[:, None]] = -math.inf
                    if case["prefix"]:
                        z = torch.cat((z, st["prefix_lse"][rows, q].double()[:, None]), 1)
                    L = torch.logsumexp(z, 1) if z.shape[1] else torch.full((z.shape[0],), -math.inf, device="cuda",
                                                                            dtype=torch.float64)
                    w = torch.exp(z - torch.where(torch.isinf(L), 0.0, L)[:, None])
                    o = w[:, :T] @ V
                    if case["prefix"]:
                        o = o + w[:, T:] * st["prefix_out"][rows, q].double()
                    out[rows, q], lse[rows, q] = o, L
    return {"out": out, "lse": lse}
