"""Cases of the operators around the sparse attention: queries and latent rows made ready and written to the paged
cache (``dsa_qk_norm_rope``), dense attention of new tokens over it (``dsa_chunk_attn``), the attention weight that
each cached position draws (``dsa_attn_weight``), and eviction by that weight (``dsa_cache_evict``).

``run`` computes an operator in its plain form (elementary torch operations in 32 bits, angles in 64, rounded once)
or, with ``own``, through the package.  ``exact`` computes it from the definition in 64 bits.
"""
import math
import random

import torch

own = False

PAGE = 64          # positions per cache page
ROW = 576          # latent row: 512 latent + 64 rotated
DV = 512
TILE = 128         # elements that share a scale in an FP8 latent row
THETA = 10000.0
EPS = 1e-6


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of a short context with 16 heads: latency of the smallest call
        dict(name="prep_token", op="prep", B=1, n0=1, n1=1, l0=4096, l1=4096, H=16, D=ROW, qn=0, kn=DV, r0=DV, R=64,
             inter=True, fp8=False, shape=0),
        # a decode step of 32 sequences, 128 heads
        dict(name="prep_batch32", op="prep", B=32, n0=1, n1=1, l0=2048, l1=4096, H=128, D=ROW, qn=0, kn=DV, r0=DV, R=64,
             inter=True, fp8=False, shape=1),
        # a prompt of 8192 tokens, queries normalised per head, FP8 latent cache
        dict(name="prep_prefill_fp8", op="prep", B=1, n0=8192, n1=8192, l0=8192, l1=8192, H=128, D=ROW, qn=DV, kn=DV,
             r0=DV, R=64, inter=False, fp8=True, shape=2),
        # indexer queries and keys of ragged chunks: 64 heads of 128, the first 64 elements rotated
        dict(name="prep_index", op="prep", B=5, n0=100, n1=333, l0=400, l1=5000, H=64, D=128, qn=128, kn=128, r0=0, R=64,
             inter=False, fp8=False, shape=3),
        # one new token of a short context, 16 heads
        dict(name="attn_token", op="attn", B=1, n0=1, n1=1, l0=4096, l1=4096, H=16, fp8=False, shape=4),
        # a decode step of 32 sequences at 32K, 128 heads
        dict(name="attn_batch32", op="attn", B=32, n0=1, n1=1, l0=32768, l1=32768, H=128, fp8=False, shape=5),
        # the last 2048 tokens of a 16K prompt
        dict(name="attn_chunk", op="attn", B=1, n0=2048, n1=2048, l0=16384, l1=16384, H=128, fp8=False, shape=6),
        # two tokens to verify for each of 8 long ragged sequences, FP8 latent cache
        dict(name="attn_ragged_fp8", op="attn", B=8, n0=2, n1=2, l0=16384, l1=131072, H=128, fp8=True, shape=7),
        # weights of a decode step of 32 sequences at 32K
        dict(name="weight_batch32", op="weight", B=32, n0=1, n1=1, l0=32768, l1=32768, H=128, fp8=False, decay=1.0,
             shape=8),
        # weights of odd chunks of new tokens, 64 heads, older weights fading
        dict(name="weight_chunk", op="weight", B=3, n0=150, n1=300, l0=5000, l1=9001, H=64, fp8=False, decay=0.5, shape=9),
        # 32 sequences of about 32K cut to 8192 positions, bf16 latent rows and index keys
        dict(name="evict_batch32", op="evict", B=32, l0=28000, l1=32768, keep=8192, sink=4, recent=512, fp8=False,
             shape=10),
        # one sequence of a million positions cut to 65536, FP8 latent rows
        dict(name="evict_1m", op="evict", B=1, l0=1048576, l1=1048576, keep=65536, sink=16, recent=4096, fp8=True,
             shape=11),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["prep", "attn", "attn", "weight", "evict"])
    shape = rng.randrange(1 << 30)
    B = _log(rng, 1, 32)
    if op == "prep":
        n1 = _log(rng, 1, max(1, 8192 // B))
        l1 = _log(rng, n1, max(n1, 16384))
        c = dict(op=op, B=B, n0=max(1, n1 // rng.choice([1, 2, 5])), n1=n1, l0=max(n1, l1 // 2), l1=l1, shape=shape)
        if rng.random() < 0.7:
            c.update(H=_log(rng, 1, 128), D=ROW, qn=rng.choice([0, DV]), kn=DV, r0=DV, R=64, fp8=rng.random() < 0.5)
        else:
            c.update(H=_log(rng, 1, 128), D=rng.choice([64, 128, 192, 256]), R=rng.choice([16, 32, 64]), fp8=False)
            c.update(qn=rng.choice([0, c["D"]]), kn=rng.choice([0, c["D"]]), r0=rng.choice([0, c["D"] - c["R"]]))
        c["inter"] = rng.random() < 0.5
        return c
    if op == "evict":
        l1 = _log(rng, 64, 1048576 // B)
        keep = _log(rng, 1, l1)
        sink = rng.randrange(0, max(1, keep // 4) + 1) if keep > 1 else 0
        recent = rng.randrange(0, max(1, keep // 4) + 1) if keep > 1 else 0
        return dict(op=op, B=B, l0=max(1, l1 // rng.choice([1, 2, 4])), l1=l1, keep=keep, sink=sink, recent=recent,
                    fp8=rng.random() < 0.5, shape=shape)
    H = rng.choice([1, 8, 16, 40, 64, 96, 128, _log(rng, 1, 128)])
    l1 = _log(rng, 1, 131072)
    B = min(B, max(1, 1048576 // l1))
    room = 128 * 2048 * 16384 // (B * H * l1)          # (token, head, position) triples of the largest listed case
    if op == "weight":
        room //= 4
    n1 = _log(rng, 1, max(1, min(l1, room, 2048)))
    c = dict(op=op, B=B, n0=max(1, n1 // rng.choice([1, 2, 5])), n1=n1, l0=max(n1, l1 // rng.choice([1, 2, 4])), l1=l1,
             H=H, fp8=rng.random() < 0.3, shape=shape)
    if op == "weight":
        c["decay"] = rng.choice([0.0, 0.5, 1.0])
    return c


def _sizes(case):
    """Cached lengths and new tokens of each sequence."""
    r = random.Random(case["shape"])
    lens = [r.randint(case["l0"], case["l1"]) for _ in range(case["B"])]
    if case["op"] == "evict":
        return lens, [1] * case["B"]
    return lens, [min(L, r.randint(case["n0"], case["n1"])) for L in lens]


def _row_bytes(fp8):
    return ROW + 20 if fp8 else 2 * ROW


def work(case):
    lens, nq = _sizes(case)
    T = sum(nq)
    if case["op"] == "prep":
        D, H = case["D"], case["H"]
        out = T * H * D * 2 + T * (_row_bytes(True) if case["fp8"] else 2 * D)
        return {"bytes": T * (H + 1) * D * 2 + out, "flops": 6 * T * (H + 1) * D}
    if case["op"] == "evict":
        kept = sum(min(L, case["keep"]) for L in lens)
        row = _row_bytes(case["fp8"]) + 256          # a latent row and its index key
        return {"bytes": sum(lens) * 4 + kept * (2 * row + 4 + 4), "flops": sum(lens)}
    H = case["H"]
    pairs = sum(n * (L - n) + n * (n + 1) // 2 for L, n in zip(lens, nq)) * H
    b = sum(lens) * _row_bytes(case["fp8"]) + T * H * (2 * ROW + 4)
    if case["op"] == "attn":
        return {"bytes": b + T * H * 2 * DV, "flops": pairs * 2 * (ROW + DV)}
    return {"bytes": b + sum(lens) * (8 if case["decay"] else 4), "flops": pairs * 2 * ROW}


# ---------------------------------------------------------------------------------------------- inputs
class State:
    pass


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape):
    """N(0, 1) in bf16, in pieces (a large cache has no room for fp32 copies)."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):
        p = flat[i:i + (1 << 27)]
        p.copy_(torch.randn(p.numel(), generator=g, device="cuda"))
    return out


def _quantise(x):
    """Latent rows as e4m3 codes (bytes) and one scale per 128 elements."""
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(*x.shape[:-1], 5, dtype=torch.float32, device=x.device)
    for i in range(0, x.shape[0], 4096):
        v = torch.nn.functional.pad(x[i:i + 4096].float(), (0, 64)).unflatten(-1, (5, TILE))
        a = v.abs().amax(-1)
        s = torch.where(a > 0, a / 448.0, torch.ones_like(a))
        scale[i:i + 4096] = s
        codes[i:i + 4096] = (v / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)[..., :ROW]
    return codes, scale


def _paging(st, lens, nq, g):
    """A batch: lengths, token offsets, a table of permuted pages, and the plain form's index tensors."""
    dev = "cuda"
    B = len(lens)
    nb = [-(-L // PAGE) for L in lens]
    st.B, st.T, st.max_len, st.max_q, st.num_blocks = B, sum(nq), max(lens), max(nq), sum(nb)
    perm = torch.randperm(st.num_blocks, generator=g, device=dev, dtype=torch.int64).int()
    table = torch.zeros(B, max(nb), dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(nb):
        table[b, :k] = perm[at:at + k]
        at += k
    st.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
    st.cu_q = torch.tensor([0] + [sum(nq[:b + 1]) for b in range(B)], dtype=torch.int32, device=dev)
    st.table = table
    st.seq = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(nq, device=dev))
    off = torch.arange(st.T, device=dev) - st.cu_q[st.seq].long()
    st.off = off
    st.pos = st.lens[st.seq].long() - torch.tensor(nq, device=dev)[st.seq] + off


def prepare(case, seed):
    g = _gen(seed)
    st = State()
    st.case = case
    lens, nq = _sizes(case)
    _paging(st, lens, nq, g)
    op = case["op"]
    if op == "prep":
        D, H = case["D"], case["H"]
        st.q = _randn(g, st.T, H, D)
        st.k = _randn(g, st.T, D) * 3
        gamma = lambda n: torch.rand(n, generator=g, device="cuda") + 0.5 if n else None  # noqa: E731
        st.qg, st.kg = gamma(case["qn"]), gamma(case["kn"])
        R = case["R"]
        st.freq = (THETA ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda()
        st.cache = _randn(g, st.num_blocks, PAGE, D)
        st.scale = None
        if case["fp8"]:
            st.cache, st.scale = _quantise(st.cache)
        return st
    if op == "evict":
        # accumulated weights: heavy-tailed, a third of the positions never attended (ties)
        w = torch.randn(st.B, st.table.shape[1] * PAGE, generator=g, device="cuda").mul_(2).exp_()
        st.weight = torch.where(torch.rand(w.shape, generator=g, device="cuda") < 0.33, torch.zeros_like(w), w)
        kv = _randn(g, st.num_blocks, PAGE, ROW)
        keys = _randn(g, st.num_blocks, PAGE, 128)
        st.arrays = [keys] + (list(_quantise(kv)) if case["fp8"] else [kv])
        nb = -(-case["keep"] // PAGE)
        st.new_table = torch.randperm(st.B * nb, generator=g, device="cuda").int().view(st.B, nb)
        st.new_arrays = [torch.zeros(st.B * nb, *a.shape[1:], dtype=a.dtype, device="cuda") for a in st.arrays]
        st.new_weight = torch.zeros(st.B, nb * PAGE, device="cuda")
        return st
    st.scale_qk = 1.0 / math.sqrt(ROW)
    st.q = _randn(g, st.T, case["H"], ROW) * 3
    st.kv = _randn(g, st.num_blocks, PAGE, ROW)
    st.kv_scale = None
    if case["fp8"]:
        st.kv, st.kv_scale = _quantise(st.kv)
    if op == "weight":
        st.start = torch.rand(st.B, st.table.shape[1] * PAGE, generator=g, device="cuda") * 4
        st.lse = _attend(st, False)
        st.weight = torch.empty_like(st.start)
    return st


# ---------------------------------------------------------------------------------------------- plain forms
def _rows(st, dtype=torch.float32):
    """Latent rows by position, [B, pages * 64, 576]."""
    x = st.kv[st.table.long()]
    if st.kv_scale is None:
        return x.to(dtype).flatten(1, 2)
    s = st.kv_scale[st.table.long()].to(dtype).repeat_interleave(TILE, dim=-1)[..., :ROW]
    return (x.view(torch.float8_e4m3fn).to(dtype) * s).flatten(1, 2)


def _logits(st, rows):
    """Scaled logits [B, max_q, H, positions], -inf where a token does not see; rows past a sequence's tokens see nothing."""
    H = st.q.shape[1]
    q = torch.zeros(st.B, st.max_q, H, ROW, dtype=rows.dtype, device="cuda")
    q[st.seq, st.off] = st.q.to(rows.dtype) * st.scale_qk
    s = torch.bmm(q.flatten(1, 2), rows.transpose(1, 2)).unflatten(1, (st.max_q, H))
    last = torch.full((st.B, st.max_q), -1, dtype=torch.int64, device="cuda")
    last[st.seq, st.off] = st.pos
    hidden = torch.arange(rows.shape[1], device="cuda") > last[:, :, None]
    return s.masked_fill_(hidden[:, :, None, :], -math.inf)


def _attend(st, values=True):
    rows = _rows(st)
    s = _logits(st, rows)
    m = s.amax(-1, keepdim=True).clamp_min(-1e30)
    p = s.sub_(m).exp_()
    l = p.sum(-1)
    lse = (m[..., 0] + l.log())[st.seq, st.off]
    if not values:
        return lse
    o = torch.bmm(p.flatten(1, 2), rows[..., :DV]).unflatten(1, p.shape[1:3]) / l[..., None]
    return o[st.seq, st.off].to(torch.bfloat16), lse


def _weigh(st):
    s = _logits(st, _rows(st))
    lse = torch.zeros(s.shape[:3], device="cuda")
    lse[st.seq, st.off] = st.lse
    add = s.sub_(lse[..., None]).exp_().sum((1, 2))
    decay = st.case["decay"]
    new = add + decay * st.weight if decay else add
    here = torch.arange(add.shape[1], device="cuda") < st.lens[:, None]
    st.weight.copy_(torch.where(here, new, st.weight))
    return st.weight


def _turn(x, gamma, cos, sin, case):
    """Norm of the leading elements, then the rotation; x [..., D], cos and sin over its pairs."""
    if gamma is not None:
        n = gamma.numel()
        h = x[..., :n]
        x = torch.cat([h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * gamma, x[..., n:]], -1)
    r0, R = case["r0"], case["R"]
    v = x[..., r0:r0 + R]
    a, b = (v[..., 0::2], v[..., 1::2]) if case["inter"] else (v[..., :R // 2], v[..., R // 2:])
    c, d = a * cos - b * sin, b * cos + a * sin
    v = torch.stack([c, d], -1).flatten(-2) if case["inter"] else torch.cat([c, d], -1)
    return torch.cat([x[..., :r0], v, x[..., r0 + R:]], -1)


def _slots(st):
    return st.table[st.seq, st.pos // PAGE].long() * PAGE + st.pos % PAGE


def _prep(st):
    c = st.case
    angle = st.pos.double()[:, None] * st.freq.double()
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _turn(st.q.float(), st.qg, cos[:, None], sin[:, None], c).to(torch.bfloat16)
    k = _turn(st.k.float(), st.kg, cos, sin, c)
    rows = st.cache.view(-1, c["D"])
    if not c["fp8"]:
        rows[_slots(st)] = k.to(torch.bfloat16)
        return q, st.cache
    v = torch.nn.functional.pad(k, (0, 64)).unflatten(-1, (5, TILE))
    a = v.abs().amax(-1)
    s = torch.where(a > 0, a / 448.0, torch.ones_like(a))
    rows[_slots(st)] = (v / s[..., None]).to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)[:, :ROW]
    st.scale.view(-1, 5)[_slots(st)] = s
    return q, st.cache.view(torch.float8_e4m3fn), st.scale


def _evict(st):
    c = st.case
    keep, W = c["keep"], st.weight.shape[1]
    pos = torch.arange(W, device="cuda")
    L = st.lens[:, None].long()
    held = (pos < c["sink"]) | (pos >= L - c["recent"])
    w = torch.where(held, torch.full_like(st.weight, math.inf), st.weight)
    w = torch.where(pos < L, w, torch.full_like(w, -math.inf))
    idx = torch.sort(w, dim=1, descending=True, stable=True).indices
    idx = torch.nn.functional.pad(idx, (0, max(0, keep - W)), value=W)[:, :keep]
    count = torch.minimum(st.lens, torch.full_like(st.lens, keep))
    rank = torch.arange(keep, device="cuda")
    there = rank < count[:, None]
    idx = torch.where(there, idx, W).sort(1).values       # ascending, the padding last
    seq = torch.arange(st.B, device="cuda")[:, None].expand_as(idx)[there]
    src = idx[there]
    dst = rank.expand_as(idx)[there]
    at = st.table[seq, src // PAGE].long() * PAGE + src % PAGE
    to = st.new_table[seq, dst // PAGE].long() * PAGE + dst % PAGE
    [n.flatten(0, 1).index_copy_(0, to, o.flatten(0, 1)[at]) for o, n in zip(st.arrays, st.new_arrays)]
    st.new_weight[seq, dst] = st.weight[seq, src]
    return _evicted(st, torch.where(there, idx, -1).int(), count)


def _evicted(st, idx, count):
    a = st.new_arrays
    rows = [a[0], a[1].view(torch.float8_e4m3fn), a[2]] if st.case["fp8"] else a
    return [idx, count, st.new_weight] + list(rows)


def run(state):
    st, op = state, state.case["op"]
    if own:
        import indexer_top_sparse_lightning_b200 as dsa
        batch = dsa.Batch(st.lens, st.cu_q, st.table, st.num_blocks, st.max_len, st.max_q)
        if op == "prep":
            q = dsa.dsa_qk_norm_rope(batch, st.freq, st.q, st.k, q_gamma=st.qg, k_gamma=st.kg, eps=EPS,
                                     rope_off=st.case["r0"], interleaved=st.case["inter"], k_cache=st.cache,
                                     k_scale=st.scale)
            return (q, st.cache) if st.scale is None else (q, st.cache.view(torch.float8_e4m3fn), st.scale)
        if op == "attn":
            return dsa.dsa_chunk_attn(batch, st.q, st.kv, st.scale_qk, kv_scale=st.kv_scale)
        if op == "weight":
            st.weight.copy_(st.start)
            return dsa.dsa_attn_weight(batch, st.q, st.kv, st.scale_qk, st.lse, st.weight, decay=st.case["decay"],
                                       kv_scale=st.kv_scale)
        idx, count = dsa.dsa_cache_evict(batch, st.weight, st.case["keep"], st.new_table, st.arrays, st.new_arrays,
                                         sink=st.case["sink"], recent=st.case["recent"], new_weight=st.new_weight)
        return _evicted(st, idx, count)
    if op == "prep":
        return _prep(st)
    if op == "attn":
        return _attend(st)
    if op == "weight":
        st.weight.copy_(st.start)
        return _weigh(st)
    return _evict(st)


# ---------------------------------------------------------------------------------------------- definitions in 64 bits
def _exact_turn(x, gamma, pos, case, freq):
    y = x.double()
    if gamma is not None:
        n = gamma.numel()
        r = (y[..., :n].square().sum(-1, keepdim=True) / n + EPS).sqrt()
        y[..., :n] = y[..., :n] / r * gamma.double()
    r0, R = case["r0"], case["R"]
    i = torch.arange(R // 2, device="cuda")
    lo, hi = (r0 + 2 * i, r0 + 2 * i + 1) if case["inter"] else (r0 + i, r0 + R // 2 + i)
    z = torch.polar(torch.ones(pos.numel(), R // 2, dtype=torch.float64, device="cuda"),
                    pos.double()[:, None] * freq.double())
    z = z.view(pos.numel(), *[1] * (y.dim() - 2), R // 2) * torch.complex(y[..., lo], y[..., hi])
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    lens, nq = _sizes(case)
    if op == "prep":
        q = _exact_turn(st.q, st.qg, st.pos, case, st.freq)
        k = _exact_turn(st.k, st.kg, st.pos, case, st.freq)
        at = _slots(st)
        if not case["fp8"]:
            cache = st.cache.double()
            cache.view(-1, case["D"])[at] = k
            return q, cache
        cache, scale = st.cache.view(torch.float8_e4m3fn).double(), st.scale.double()
        for t in range(5):
            g = k[:, t * TILE:(t + 1) * TILE]
            a = g.abs().amax(-1, keepdim=True)
            s = torch.where(a > 0, a / 448, torch.ones_like(a))
            cache.view(-1, ROW)[at, t * TILE:(t + 1) * TILE] = g / s
            scale.view(-1, 5)[at, t] = s[:, 0]
        return q, cache, scale
    if op == "evict":
        return None          # choices and copies: nothing is computed
    H = case["H"]
    if sum(n * L for n, L in zip(nq, lens)) * H > 6e9:
        return None
    outs, lses, start = [], [], 0
    if op == "weight":
        w = st.start.double()
    for b, (L, n) in enumerate(zip(lens, nq)):
        pages = st.table[b, :-(-L // PAGE)].long()
        x = st.kv[pages]
        if st.kv_scale is None:
            x = x.double()
        else:
            f = torch.arange(ROW, device="cuda") // TILE
            x = x.view(torch.float8_e4m3fn).double() * st.kv_scale[pages].double()[..., f]
        x = x.reshape(-1, ROW)[:L]
        step = max(1, (1 << 28) // (H * L))
        if op == "weight":
            w[b, :L] *= case["decay"]
        for j in range(0, n, step):
            m = min(step, n - j)
            t = slice(start + j, start + j + m)
            s = (st.q[t].double().reshape(m * H, ROW) @ x.T * st.scale_qk).view(m, H, L)
            p = torch.arange(L - n + j, L - n + j + m, device="cuda")
            s.masked_fill_((torch.arange(L, device="cuda") > p[:, None])[:, None], -math.inf)
            if op == "weight":
                w[b, :L] += (s - st.lse[t].double()[..., None]).exp().sum((0, 1))
                continue
            lse = torch.logsumexp(s, -1)
            outs.append(((s - lse[..., None]).exp().view(m * H, L) @ x[:, :DV]).view(m, H, DV))
            lses.append(lse)
        start += n
    return w if op == "weight" else (torch.cat(outs), torch.cat(lses))
