"""The operators around a paged key/value cache, as cases that can be measured.

* rotate -- the position rotation of queries and keys in the prefill layout
  [b, heads, n, d], and its gradient (the inverse rotation).
* append -- the keys and values of new tokens written into the pages of a chunk
  cache, the keys (and the queries handed over with them) rotated by their
  position on the way; the pages that a call fills are listed.
* dense  -- attention of one new token per sequence over every key of its paged
  cache (or over its last window of chunks).

`run` computes an operator in its plain form from elementary torch operations, or,
where `own` is true, with the framework's calls.
"""
import math

import numpy as np
import torch

own = False

CHUNK = 64          # keys per page
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases ------------------------------------------------------------------
def listed():
    return [
        # one conversation, a short context: latency of a single step (7B-shaped heads)
        dict(name="dense_chat", op="dense", dtype="bf16", batch=1, heads_q=32, heads_kv=8, d=128, max_len=1013,
             spread=False, window=0),
        # a full batch of long contexts, one key head per query head (the decode workload's shape)
        dict(name="dense_32k", op="dense", dtype="bf16", batch=8, heads_q=16, heads_kv=16, d=64, max_len=32768,
             spread=False, window=0),
        # a serving batch: lengths from nothing to 16K, idle slots among them
        dict(name="dense_ragged", op="dense", dtype="bf16", batch=33, heads_q=32, heads_kv=8, d=128, max_len=16384,
             spread=True, window=0),
        # one very long document, its last page partly filled
        dict(name="dense_512k", op="dense", dtype="bf16", batch=1, heads_q=32, heads_kv=8, d=128, max_len=524225,
             spread=False, window=0),
        # a sliding-window layer in fp32
        dict(name="dense_window_f32", op="dense", dtype="f32", batch=7, heads_q=8, heads_kv=2, d=64, max_len=4001,
             spread=True, window=512),
        # one decode step of a full batch, far positions: a few hundred KB, latency
        dict(name="append_step", op="append", dtype="bf16", batch=64, heads_q=32, heads_kv=8, d=128, new=1,
             layout="packed", max_len=500000, rotary=128, interleaved=False),
        # packed prompts of different lengths, sliced from one fused projection
        dict(name="append_prompts", op="append", dtype="bf16", batch=16, heads_q=32, heads_kv=8, d=128, new=3001,
             layout="packed", max_len=8192, rotary=128, interleaved=False),
        # a right-padded batch in the prefill layout, half the head rotated, pairs interleaved
        dict(name="append_padded_f32", op="append", dtype="f32", batch=3, heads_q=4, heads_kv=2, d=64, new=777,
             layout="padded", max_len=2000, rotary=32, interleaved=True),
        # queries and keys of the 345M-shaped prefill, sliced from one fused projection
        dict(name="rotate_345m", op="rotate", dtype="bf16", batch=4, heads_q=16, heads_kv=16, d=64, n=8192,
             positions="", rotary=64, interleaved=False, inverse=False),
        # the fp32 gradients of a 16K training step, rotated back
        dict(name="rotate_grad_16k", op="rotate", dtype="f32", batch=2, heads_q=16, heads_kv=16, d=128, n=16384,
             positions="", rotary=128, interleaved=False, inverse=True),
        # a short continuation at far positions of its own, half the head rotated
        dict(name="rotate_far", op="rotate", dtype="bf16", batch=1, heads_q=8, heads_kv=2, d=128, n=257,
             positions="row", rotary=64, interleaved=True, inverse=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    d = rng.choice([64, 128])
    g = rng.choice([1, 2, 4, 8, 16])
    h = g * rng.choice([1, 2, 4, 8] if g <= 4 else [1, 2, 4])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    size = 2 if dtype == "bf16" else 4
    op = rng.choice(["dense", "dense", "append", "rotate"])
    if op == "dense":
        batch = _log(rng, 1, 96)
        most = min(500000, (1 << 30) // (batch * g * d * size * 2))
        return dict(op=op, dtype=dtype, batch=batch, heads_q=h, heads_kv=g, d=d, max_len=_log(rng, 17, most),
                    spread=rng.random() < 0.7, window=rng.choice([0, 0, 0, 64, 192, 512, 4096]))
    rotary = rng.choice([16, 32, 64, d])
    inter = rng.random() < 0.5
    if op == "append":
        layout = rng.choice(["packed", "padded"])
        batch = _log(rng, 1, 128)
        most = (1 << 28) // (batch * (h + 2 * g) * d * size)
        new = rng.choice([1, _log(rng, 1, max(2, min(4000, most)))])
        return dict(op=op, dtype=dtype, batch=batch, heads_q=h, heads_kv=g, d=d, new=new, layout=layout,
                    max_len=new + _log(rng, 1, 400000), rotary=rotary, interleaved=inter)
    batch = _log(rng, 1, 8)
    most = min(20000, (1 << 28) // (batch * (h + g) * d * size))
    return dict(op=op, dtype=dtype, batch=batch, heads_q=h, heads_kv=g, d=d, n=_log(rng, 5, most),
                positions=rng.choice(["", "shared", "row"]), rotary=rotary, interleaved=inter,
                inverse=rng.random() < 0.5)


def _lengths(case):
    """Cache length of each sequence: the longest first; where they spread, an idle slot
    among three or more and the others anywhere up to the longest."""
    b, m = case["batch"], case["max_len"]
    if case["op"] == "append":  # room for the new tokens
        return [max(n, 1 + int(m * (((i + 1) * 0.6180339887) % 1.0))) for i, n in enumerate(_new_counts(case))]
    if not case["spread"]:
        return [m] * b
    lens = [1 + int((m - 1) * (((i + 1) * 0.6180339887) % 1.0)) for i in range(b)]
    lens[0] = m
    if b >= 3:
        lens[1] = 0
    return lens


def _new_counts(case):
    """New tokens of each sequence: the longest first, an idle slot among three or more."""
    b, m = case["batch"], case["new"]
    if m == 1:
        return [1] * b
    n = [1 + int((m - 1) * (((i + 1) * 0.7548776662) % 1.0)) for i in range(b)]
    n[0] = m
    if b >= 3:
        n[2] = 0
    return n


def _first_chunk(case, length):
    """First chunk that a new token at the end of `length` keys attends to."""
    own_chunk = max(0, length - 1) // CHUNK
    w = case["window"] // CHUNK
    return 0 if w == 0 else max(0, own_chunk + 1 - w)


def work(case):
    size = 2 if case["dtype"] == "bf16" else 4
    b, h, g, d = case["batch"], case["heads_q"], case["heads_kv"], case["d"]
    if case["op"] == "dense":
        keys = sum(max(0, n - CHUNK * _first_chunk(case, n)) for n in _lengths(case))
        pages = sum(-(-n // CHUNK) - _first_chunk(case, n) for n in _lengths(case) if n)
        return {"bytes": 2 * keys * g * d * size + 2 * b * h * d * size + 4 * b * h + 4 * b + 4 * pages,
                "flops": 4 * keys * h * d}
    if case["op"] == "append":
        t = sum(_new_counts(case))
        return {"bytes": 2 * t * (h + 2 * g) * d * size + 8 * b + 4 * t, "flops": 3 * t * (h + g) * case["rotary"]}
    t = b * case["n"]
    return {"bytes": 2 * t * (h + g) * d * size + (4 * t if case["positions"] else 0),
            "flops": 3 * t * (h + g) * case["rotary"]}


# ---- inputs -----------------------------------------------------------------
def _randn(gen, *shape, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    flat = out.view(-1)
    for i in range(0, flat.numel(), 1 << 27):  # drawn in fp32 slabs, rounded once
        part = flat[i:i + (1 << 27)]
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda"))
    return out


def _inv_freq(case):
    r = case["rotary"]
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def _tables(lens, first, max_chunks, seed):
    """A pool just large enough, its pages dealt out in a shuffled order; -1 where a
    sequence holds no page (before `first`, after its end)."""
    counts = [max(0, -(-n // CHUNK) - f) for n, f in zip(lens, first)]
    pool = sum(counts) + 3
    perm = np.random.RandomState(seed % (1 << 31)).permutation(pool).astype(np.int32)
    table = np.full((len(lens), max_chunks), -1, np.int32)
    at = 0
    for i, (c, f) in enumerate(zip(counts, first)):
        table[i, f:f + c] = perm[at:at + c]
        at += c
    return table, pool


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dtype = DTYPES[case["dtype"]]
    b, h, g, d = case["batch"], case["heads_q"], case["heads_kv"], case["d"]
    s = {"case": dict(case), "op": case["op"]}
    if case["op"] == "dense":
        lens = _lengths(case)
        max_chunks = max(1, -(-max(lens) // CHUNK))
        table, pool = _tables(lens, [0] * b, max_chunks, seed)
        q = _randn(gen, b, h, d, dtype=dtype)
        k = _randn(gen, pool, g, CHUNK, d, dtype=dtype)
        v = _randn(gen, pool, g, CHUNK, d, dtype=dtype)
        # each key head of each sequence remembers a few keys its query looks for
        rng = np.random.RandomState(seed % (1 << 31))
        for _ in range(4):
            at = [(i, j, int(rng.randint(n))) for i, n in enumerate(lens) if n for j in range(g)]
            if at:
                bi, gi, pos = (torch.tensor(x, device="cuda") for x in zip(*at))
                page = torch.tensor([int(table[i, p // CHUNK]) for i, _, p in at], device="cuda")
                row = q[bi, gi * (h // g)].float()
                k[page, gi, pos % CHUNK] = (8.0 * row / row.norm(dim=-1, keepdim=True)).to(dtype)
        s.update(q=q, k_pages=k, v_pages=v, block_table=torch.from_numpy(table).cuda(),
                 seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_chunks=max_chunks)
        s.update(out=torch.empty_like(q), lse=torch.empty(b, h, device="cuda"))
        if own:
            import chunk_wise_hierarchical_b200 as hils
            s["call"] = hils.DenseDecode(b, h, g, d, max_chunks, dtype, window=case["window"])
        return s
    s["inv_freq"] = _inv_freq(case)
    if case["op"] == "append":
        new, lens = _new_counts(case), _lengths(case)
        max_chunks = max(1, -(-max(lens) // CHUNK))
        # the pool of a window layer: pages before the new tokens were handed back
        table, pool = _tables(lens, [(n - c) // CHUNK for n, c in zip(lens, new)], max_chunks, seed)
        if case["layout"] == "packed":
            t = sum(new)
            fused = _randn(gen, t, h + 2 * g, d, dtype=dtype)
            s["cu_new"] = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
            s["q"], s["k"], s["v"] = fused[:, :h], fused[:, h:h + g], fused[:, h + g:]
            s["q_out"] = torch.empty(t, h, d, dtype=dtype, device="cuda")
            slots = b + t // CHUNK
        else:
            n = case["new"]
            s["new_lens"] = torch.tensor(new, dtype=torch.int32, device="cuda")
            s["q"], s["k"], s["v"] = (_randn(gen, b, x, n, d, dtype=dtype) for x in (h, g, g))
            s["q_out"] = torch.zeros(b, h, n, d, dtype=dtype, device="cuda")
            slots = b + b * n // CHUNK
        s.update(k_pages=_randn(gen, pool, g, CHUNK, d, dtype=dtype), v_pages=_randn(gen, pool, g, CHUNK, d, dtype=dtype),
                 block_table=torch.from_numpy(table).cuda(),
                 seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda"),
                 full_pages=torch.empty(slots, dtype=torch.int32, device="cuda"), max_chunks=max_chunks)
        if own:
            import chunk_wise_hierarchical_b200 as hils
            s["call"] = hils.Append(b, h, g, d, max_chunks, dtype, inv_freq=s["inv_freq"],
                                    interleaved=case["interleaved"])
        return s
    n = case["n"]
    if case["inverse"]:  # gradients as the backward pass writes them
        s["q"], s["k"] = _randn(gen, b, h, n, d, dtype=dtype), _randn(gen, b, g, n, d, dtype=dtype)
    else:                # slices of one fused projection [b, n, heads, d]
        fused = _randn(gen, b, n, h + 2 * g, d, dtype=dtype)
        s["q"], s["k"] = fused[:, :, :h].transpose(1, 2), fused[:, :, h:h + g].transpose(1, 2)
    s["positions"] = None
    if case["positions"]:
        shape = (n,) if case["positions"] == "shared" else (b, n)
        s["positions"] = torch.randint(0, 4 << 20, shape, generator=gen, device="cuda", dtype=torch.int32)
    s["q_out"] = torch.empty(b, h, n, d, dtype=dtype, device="cuda")
    s["k_out"] = torch.empty(b, g, n, d, dtype=dtype, device="cuda")
    if own:
        import chunk_wise_hierarchical_b200 as hils
        s["call"] = hils.rotate
    return s


# ---- the framework's calls --------------------------------------------------
def _run_own(s):
    if s["op"] == "dense":
        s["call"](s["q"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], out=s["out"], lse=s["lse"])
        return {"out": s["out"], "lse": s["lse"]}
    if s["op"] == "append":
        s["call"](s["k"], s["v"], s["k_pages"], s["v_pages"], s["block_table"], s["seq_lens"], q=s["q"],
                  q_out=s["q_out"], cu_new=s.get("cu_new"), new_lens=s.get("new_lens"), full_pages=s["full_pages"])
        return {n: s[n] for n in ("q_out", "k_pages", "v_pages", "full_pages")}
    c = s["case"]
    q, k = s["call"](s["q"], s["inv_freq"], k=s["k"], positions=s["positions"], inverse=c["inverse"],
                     interleaved=c["interleaved"], q_out=s["q_out"], k_out=s["k_out"])
    return {"q": q, "k": k}


# ---- the plain forms --------------------------------------------------------
def _turn(x, pos, inv_freq, interleaved, inverse=False):
    """x [..., d] rotated by the angles pos * inv_freq (pos: the shape that broadcasts to x's
    leading dimensions); angles in 64 bits, products in 32."""
    ang = pos.double().unsqueeze(-1) * inv_freq.double()
    c, w = ang.cos().float(), ang.sin().float()
    if inverse:
        w = -w
    r = 2 * inv_freq.numel()
    x = x.float()
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., :r // 2], x[..., r // 2:r])
    lo, hi = a * c - b * w, b * c + a * w
    both = torch.stack((lo, hi), -1).flatten(-2) if interleaved else torch.cat((lo, hi), -1)
    return torch.cat((both, x[..., r:]), -1)


def _plain_dense(s):
    c = s["case"]
    q, table, lens = s["q"], s["block_table"], s["seq_lens"].long()
    b, h, d = q.shape
    g = c["heads_kv"]
    pages = table.clamp(min=0).long()
    k, v = s["k_pages"][pages].float(), s["v_pages"][pages].float()              # [b, C, g, 64, d]
    score = torch.matmul(q.float().view(b, 1, g, h // g, d), k.transpose(-1, -2)) / math.sqrt(d)
    pos = torch.arange(table.shape[1] * CHUNK, device=q.device).view(1, -1, 1, 1, CHUNK)
    n = lens.view(b, 1, 1, 1, 1)
    seen = pos < n
    if c["window"]:
        seen = seen & (pos >= ((n - 1) // CHUNK + 1 - c["window"] // CHUNK) * CHUNK)
    score = score.masked_fill(~seen, -math.inf)                                   # [b, C, g, G, 64]
    top = score.amax(dim=(1, 4), keepdim=True)
    p = torch.exp(score - top.clamp(min=-3e38))
    mass = p.sum(dim=(1, 4))                                                      # [b, g, G]
    out = torch.matmul(p, v).sum(dim=1) / mass.clamp(min=1e-38).unsqueeze(-1)
    lse = top.view(b, g, h // g) + torch.log(mass)
    return {"out": out.reshape(b, h, d).to(q.dtype), "lse": lse.reshape(b, h)}


def _plain_append(s):
    c = s["case"]
    q, k, v, table = s["q"], s["k"], s["v"], s["block_table"].long()
    lens = s["seq_lens"].long()
    if "cu_new" in s:
        cu = s["cu_new"].long()
        t = torch.arange(k.shape[0], device=k.device)
        seq = torch.searchsorted(cu, t, right=True) - 1
        count, start = cu[1:] - cu[:-1], cu[:-1]
        pos = lens[seq] - count[seq] + (t - cu[seq])
        s["q_out"].copy_(_turn(q, pos[:, None], s["inv_freq"], c["interleaved"]))
        kr, vr = _turn(k, pos[:, None], s["inv_freq"], c["interleaved"]).to(k.dtype), v
    else:
        b, _, n, _ = k.shape
        count, start = s["new_lens"].long(), torch.arange(b, device=k.device) * n
        i = torch.arange(n, device=k.device).expand(b, n)
        at = (lens - count)[:, None] + i
        valid = i < count[:, None]
        turned = _turn(q, at[:, None], s["inv_freq"], c["interleaved"]).to(q.dtype)
        s["q_out"].copy_(torch.where(valid[:, None, :, None], turned, s["q_out"]))
        seq, tok = valid.nonzero(as_tuple=True)
        pos = at[seq, tok]
        kr = _turn(k, at[:, None], s["inv_freq"], c["interleaved"]).to(k.dtype)[seq, :, tok]
        vr = v[seq, :, tok]
    page = table[seq, pos // CHUNK]
    s["k_pages"][page, :, pos % CHUNK] = kr
    s["v_pages"][page, :, pos % CHUNK] = vr
    # slot b + start // 64 + j: the j-th page that sequence b filled
    s["full_pages"].fill_(-1)
    full = pos % CHUNK == CHUNK - 1
    first = ((lens - count) // CHUNK)[seq]
    slot = seq + start[seq] // CHUNK + pos // CHUNK - first
    s["full_pages"][slot[full]] = page[full].int()
    return {n: s[n] for n in ("q_out", "k_pages", "v_pages", "full_pages")}


def _plain_rotate(s):
    c = s["case"]
    n = s["q"].shape[2]
    pos = torch.arange(n, device=s["q"].device) if s["positions"] is None else s["positions"]
    pos = pos.view(-1, 1, n)
    for x, out in ((s["q"], s["q_out"]), (s["k"], s["k_out"])):
        out.copy_(_turn(x, pos, s["inv_freq"], c["interleaved"], c["inverse"]))
    return {"q": s["q_out"], "k": s["k_out"]}


def run(state):
    if own:
        return _run_own(state)
    return {"dense": _plain_dense, "append": _plain_append, "rotate": _plain_rotate}[state["op"]](state)


# ---- the definitions in 64 bits ---------------------------------------------
def _spin(x, pos, inv_freq, interleaved, sign=1.0):
    """Each pair as one complex number times exp(i * pos * frequency); x [n, heads, d], pos [n]."""
    r = 2 * inv_freq.numel()
    out = x.double().clone()
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       sign * pos.double()[:, None, None] * inv_freq.double())
    even, odd = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    z = torch.complex(out[..., even].contiguous(), out[..., odd].contiguous()) * turn
    out[..., even], out[..., odd] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dense":
        b, h, g, d = case["batch"], case["heads_q"], case["heads_kv"], case["d"]
        out = torch.zeros(b, h, d, dtype=torch.float64, device="cuda")
        lse = torch.full((b, h), -math.inf, dtype=torch.float64, device="cuda")
        for i, n in enumerate(_lengths(case)):
            if n == 0:
                continue
            lo = CHUNK * _first_chunk(case, n)
            pages = s["block_table"][i, lo // CHUNK:-(-n // CHUNK)].long()
            for j in range(g):
                k = s["k_pages"][pages, j].double().reshape(-1, d)[:n - lo]
                v = s["v_pages"][pages, j].double().reshape(-1, d)[:n - lo]
                rows = slice(j * (h // g), (j + 1) * (h // g))
                x = s["q"][i, rows].double() @ k.T * d ** -0.5
                lse[i, rows] = torch.logsumexp(x, -1)
                out[i, rows] = torch.exp(x - lse[i, rows, None]) @ v
        return {"out": out, "lse": lse}
    if case["op"] == "append":
        q_out, kp, vp = (s[n].double() for n in ("q_out", "k_pages", "v_pages"))
        full = torch.full_like(s["full_pages"], -1)
        at = 0
        for i, (new, n) in enumerate(zip(_new_counts(case), _lengths(case))):
            pos = torch.arange(n - new, n, device="cuda")
            packed = case["layout"] == "packed"
            q, k, v = ((s[x][at:at + new] if packed else s[x][i, :, :new].transpose(0, 1)) for x in "qkv")
            page = s["block_table"][i].long()[pos // CHUNK]
            turned = _spin(q, pos, s["inv_freq"], case["interleaved"])
            if packed:
                q_out[at:at + new] = turned
            else:
                q_out[i, :, :new] = turned.transpose(0, 1)
            kp[page, :, pos % CHUNK] = _spin(k, pos, s["inv_freq"], case["interleaved"])
            vp[page, :, pos % CHUNK] = v.double()
            slot = i + at // CHUNK
            ends = page[pos % CHUNK == CHUNK - 1].int()
            # the first page that can fill is the one the first new token goes to
            full[slot:slot + len(ends)] = ends
            at += new if packed else case["new"]
        # rows that are not written hold whatever the caller's buffer held
        return {"q_out": q_out, "k_pages": kp, "v_pages": vp, "full_pages": full}
    n = case["n"]
    sign = -1.0 if case["inverse"] else 1.0
    got = {}
    for name in "qk":
        rows = []
        for i in range(case["batch"]):
            pos = s["positions"]
            pos = torch.arange(n, device="cuda") if pos is None else pos if pos.dim() == 1 else pos[i]
            rows.append(_spin(s[name][i].transpose(0, 1), pos, s["inv_freq"], case["interleaved"], sign).transpose(0, 1))
        got[name] = torch.stack(rows)
    return got
