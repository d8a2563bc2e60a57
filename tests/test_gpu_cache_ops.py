"""The paged-cache operators on the GPU against their fp64 oracle.

Tolerances, derived from the arithmetic (u(t) = eps(t) / 2, half a step of the output type):
* rotate: the output is x cos - y sin in fp32, rounded once.  The angle's remainder is rounded
  to fp32 once (pi * 2^-24 at most), sincospif is good to 2 ulp of 1, the products and the sum
  round three times: the value is off by at most (|x| + |y|) 2^-20, then u(out) relative.
* dense: fp32 sums of d products are off by d 2^-23 sum |q||k| scale =: e_s (2^-23: a tensor
  core may truncate); exp and the split of p into two bf16 parts add 2^-16 relative; the sums
  over n keys n 2^-24.  So each p is off by r = 2 e_s + 2^-16 + n 2^-23 relative (twice e_s:
  the logit and the normaliser), the output by r sum_j p_j |v_j| + u(out) |out|, the
  log-sum-exp by r + 2^-22 |lse|.
  (The weights now enter in three parts that hold them: 2^-16 is wider than it need be, and the
  cases at the end on weights and sums are held to less.)
"""
import ctypes
import math

import numpy as np
import pytest
import torch

import chunk_wise_hierarchical_b200 as hils
from oracle import cache_oracle as CO
from oracle import hils_oracle as O
from parity_util import check_close

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _np(t):
    return t.detach().double().cpu().numpy()


def _u(dtype):
    return torch.finfo(dtype).eps / 2


def _randn(*shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def _freq(r):
    return (10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64) / r)).float().cuda()


def _close(got, want, bound, what=""):
    got = _np(got) if torch.is_tensor(got) else got
    assert got.shape == want.shape
    assert np.array_equal(np.isfinite(got), np.isfinite(want)), what + ": finite values elsewhere"
    fin = np.isfinite(want)
    err = np.abs(got - np.where(fin, want, 0))[fin]
    over = err - np.broadcast_to(bound, want.shape)[fin]
    assert err.size == 0 or over.max() <= 0, f"{what}: off by {err[over.argmax()]:.3g}, {over.max():.3g} over its bound"


# ---- rotate -----------------------------------------------------------------
def _rotate_bound(x, want, out_dtype, rot, interleaved):
    a = np.abs(x)
    mag = np.zeros_like(a)
    if interleaved:
        pair = a[..., 0:rot:2] + a[..., 1:rot:2]
        mag[..., 0:rot:2] = mag[..., 1:rot:2] = pair
    else:
        pair = a[..., :rot // 2] + a[..., rot // 2:rot]
        mag[..., :rot // 2] = mag[..., rot // 2:rot] = pair
    e = mag * 2.0 ** -20
    return e + _u(out_dtype) * (np.abs(want) + e)


@pytest.mark.parametrize("dtype,out_dtype", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("d,rot,inter", [(64, 64, False), (64, 16, True), (128, 128, True), (128, 96, False)])
@pytest.mark.parametrize("b,h,g,n,pos", [(1, 1, 1, 1, None), (2, 8, 2, 37, "row"), (3, 4, 4, 65, "shared")])
def test_rotate_matches_oracle(dtype, out_dtype, d, rot, inter, b, h, g, n, pos):
    dt, od = DT[dtype], DT[out_dtype]
    fused = _randn(b, n, h + 2 * g, d, dtype=dt, seed=b + d)
    q, k = fused[:, :, :h].transpose(1, 2), fused[:, :, h:h + g].transpose(1, 2)
    p = None
    if pos:  # far positions, the largest int32 and negative ones among them
        gen = torch.Generator().manual_seed(5)
        p = torch.randint(0, 1 << 23, (n,) if pos == "shared" else (b, n), generator=gen, dtype=torch.int32)
        p.view(-1)[0], p.view(-1)[-1] = 2**31 - 1, -12345
    f = _freq(rot)
    for inverse in (False, True):
        qo = torch.full((b, h, n, d), 7.0, dtype=od, device="cuda")
        ko = torch.full((b, g, n, d), 7.0, dtype=od, device="cuda")
        hils.rotate(q, f, k=k, positions=None if p is None else p.cuda(), inverse=inverse, interleaved=inter,
                    q_out=qo, k_out=ko)
        for x, o in ((q, qo), (k, ko)):
            want = CO.rotate(_np(x), _np(f), None if p is None else p.numpy(), inter, inverse)
            _close(o, want, _rotate_bound(_np(x), want, od, rot, inter), "rotate")


@pytest.mark.parametrize("inter", [False, True])
def test_rotate_copies_what_lies_behind_the_rotated_part(inter):
    """Bit for bit, whatever it is (an infinity beside a number among it)."""
    for dt in DT.values():
        x = _randn(1, 2, 40, 64, dtype=dt, seed=8)
        x[..., 33::2], x[0, 0, 5, 40], x[0, 1, 7, 50] = -math.inf, math.nan, -0.0
        y = hils.rotate(x, _freq(32), interleaved=inter)
        bits = torch.int16 if dt == torch.bfloat16 else torch.int32
        assert torch.equal(y[..., 32:].view(bits), x[..., 32:].view(bits))
        assert torch.isfinite(y[..., :32]).all()


def test_rotate_beyond_32_bit_offsets():
    """Rows whose element offsets pass 2^31, in place, at positions of their own index."""
    n, d = (1 << 24) + 5, 128
    x = torch.empty(1, 1, n, d, dtype=torch.bfloat16, device="cuda")
    tail = _randn(1, 1, 9, d, dtype=torch.bfloat16, seed=50)
    x[:, :, -9:] = tail
    f = _freq(d)
    hils.rotate(x, f, q_out=x)
    want = CO.rotate(_np(tail), _np(f), list(range(n - 9, n)))
    _close(x[:, :, -9:], want, _rotate_bound(_np(tail), want, torch.bfloat16, d, False), "rotate")


def test_rotate_in_place_and_alone():
    q = _randn(2, 4, 130, 64, dtype=torch.bfloat16, seed=0)
    f = _freq(64)
    want = hils.rotate(q, f)
    assert torch.equal(hils.rotate(q.clone(), f, q_out=None), want)
    x = q.clone()
    assert hils.rotate(x, f, q_out=x) is x and torch.equal(x, want)
    # a slice of a fused projection, in place: the other slices stay
    fused = _randn(2, 130, 12, 64, dtype=torch.bfloat16, seed=1)
    ref = fused.clone()
    s = fused[:, :, :4].transpose(1, 2)
    r = hils.rotate(s, f)
    hils.rotate(s, f, q_out=s)
    assert torch.equal(s, r) and torch.equal(fused[:, :, 4:], ref[:, :, 4:])
    assert hils.rotate(q[:, :, :0], f).shape == (2, 4, 0, 64)
    assert hils.rotate(q[:0], f).shape == (0, 4, 130, 64)


def test_rotate_inverse_is_the_gradient():
    """L = sum(y * rotate(x)) is linear in x: its gradient is rotate^-1(y), checked against the
    formula and against differences of the oracle's L."""
    b, h, n, d, rot = 1, 2, 9, 64, 32
    x, y = _randn(b, h, n, d, dtype=torch.float32, seed=3), _randn(b, h, n, d, dtype=torch.float32, seed=4)
    f = _freq(rot)
    for inter in (False, True):
        grad = _np(hils.rotate(y, f, inverse=True, interleaved=inter))
        rng = np.random.default_rng(0)
        for _ in range(12):
            at = tuple(rng.integers(0, s) for s in x.shape)
            step = np.zeros(x.shape)
            step[at] = 0.5
            lo, hi = (np.sum(_np(y) * CO.rotate(_np(x) + s * step, _np(f), None, inter)) for s in (-1, 1))
            assert abs((hi - lo) - grad[at]) <= 8 * 2.0 ** -20
        # and it undoes the rotation: two roundings of the same bound
        back = hils.rotate(hils.rotate(x, f, interleaved=inter), f, inverse=True, interleaved=inter)
        _close(back, _np(x), 3 * _rotate_bound(_np(x), _np(x), torch.float32, rot, inter) + 2.0 ** -19, "round trip")


# ---- append -----------------------------------------------------------------
def _table(lens, max_chunks, pool, seed):
    perm = np.random.RandomState(seed).permutation(pool)
    t = np.full((len(lens), max_chunks), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        c = -(-n // 64)
        t[b, :c] = perm[at:at + c]
        at += c
    assert at <= pool
    return t


def _append_check(layout, counts, lens, h, g, d, dtype, rot, inter, with_q=True, pad_rows=0, spoil=None):
    dt = DT[dtype]
    b = len(counts)
    max_chunks = max(1, -(-max(lens) // 64))
    pool = sum(-(-n // 64) for n in lens) + 2
    table = _table(lens, max_chunks, pool, seed=1)
    if spoil:
        spoil(table)
    kp, vp = _randn(pool, g, 64, d, dtype=dt, seed=2), _randn(pool, g, 64, d, dtype=dt, seed=3)
    kp0, vp0 = kp.clone(), vp.clone()
    f = _freq(rot) if rot else None
    call = hils.Append(b, h, g, d, max_chunks, dt, inv_freq=f, interleaved=inter)
    kw = {}
    if layout == "packed":
        cu = np.concatenate([[0], np.cumsum(counts)])
        t = int(cu[-1]) + pad_rows
        fused = _randn(t, h + 2 * g, d, dtype=dt, seed=4)
        q, k, v = fused[:, :h], fused[:, h:h + g], fused[:, h + g:]
        kw["cu_new"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        row = lambda x, bi, i: _np(x[int(cu[bi]) + i])
        at = lambda bi, i: int(cu[bi]) + i
        start = lambda bi: int(cu[bi])
        tokens = t
    elif layout == "single":
        assert all(c == 1 for c in counts)
        fused = _randn(b, h + 2 * g, d, dtype=dt, seed=4)
        q, k, v = fused[:, :h], fused[:, h:h + g], fused[:, h + g:]
        row = lambda x, bi, i: _np(x[bi])
        at = lambda bi, i: bi
        start = lambda bi: bi
        tokens = b
    else:
        n = max(counts) + pad_rows
        q, k, v = (_randn(b, x, n, d, dtype=dt, seed=4 + x) for x in (h, g, g + 100))
        v = v[:, :g]  # strides of its own
        if min(counts) < n:
            kw["new_lens"] = torch.tensor(counts, dtype=torch.int32, device="cuda")
        row = lambda x, bi, i: _np(x[bi, :, i])
        at = lambda bi, i: (bi, slice(None), i)
        start = lambda bi: bi * n
        tokens = b * n
    q_out = torch.full(q.shape, 7.0, dtype=dt, device="cuda") if with_q else None
    full = torch.full((hils.append_slots(b, tokens),), 99, dtype=torch.int32, device="cuda")
    call(k, v, kp, vp, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
         q=q if with_q else None, q_out=q_out, full_pages=full, **kw)
    status = call.device_status()
    q_rows, wk, wv, filled = CO.append(
        lambda bi, i: (row(q, bi, i) if with_q else None, row(k, bi, i), row(v, bi, i)),
        _np(kp0), _np(vp0), table, lens, counts, None if f is None else _np(f), inter)
    assert torch.equal(vp, torch.from_numpy(wv).to(dt).cuda()), "values are copied"
    keys = np.abs(_np(kp0)).max()
    changed = np.abs(wk - _np(kp0)) > 0
    assert np.array_equal(_np(kp)[~changed], _np(kp0)[~changed]), "untouched rows stay"
    mag = max(keys, np.abs(_np(k)).max() if k.numel() else 0)
    _close(kp, wk, np.where(changed, 2 * mag * 2.0 ** -20 * (1 + _u(dt)) + _u(dt) * np.abs(wk), 0), "k_pages")
    if with_q:
        got = _np(q_out)
        want = np.full(got.shape, 7.0)
        for (bi, i), x in q_rows.items():
            want[at(bi, i)] = x
        qm = np.abs(_np(q)).max() if q.numel() else 0
        _close(got, want, np.where(want == 7.0, 0, 2 * qm * 2.0 ** -20 * 2 + _u(dt) * np.abs(want)), "q_out")
    got = full.cpu().numpy()
    want = np.full(got.shape, -1)
    for bi, pages in enumerate(filled):
        s0 = bi + start(bi) // 64
        want[s0:s0 + len(pages)] = pages
    assert np.array_equal(got, want), "full_pages"
    return status


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,h,g,rot,inter", [(64, 2, 2, 64, False), (128, 8, 2, 128, False), (128, 8, 1, 32, True),
                                             (64, 4, 1, 0, False)])
@pytest.mark.parametrize("layout,counts,lens", [
    ("single", [1, 1, 1, 1], [1, 64, 65, 1000]),
    ("packed", [1], [1]),
    ("packed", [64, 0, 130, 1, 0, 63], [64, 10, 200, 128, 0, 127]),
    ("padded", [70, 0, 33], [70, 5, 161]),
    ("padded", [5, 5], [5, 69]),
])
def test_append_matches_oracle(dtype, d, h, g, rot, inter, layout, counts, lens):
    assert _append_check(layout, counts, lens, h, g, d, dtype, rot, inter) == 0


def test_append_without_queries_and_with_padding_rows():
    assert _append_check("packed", [3, 70], [3, 70], 2, 2, 64, "bf16", 64, False, with_q=False, pad_rows=9) == 0
    assert _append_check("packed", [3, 70], [3, 70], 2, 2, 64, "bf16", 64, False, pad_rows=100) == 0
    assert _append_check("padded", [3, 70], [3, 70], 2, 2, 64, "bf16", 64, False, pad_rows=30) == 0
    assert _append_check("packed", [0, 0], [3, 0], 2, 2, 64, "f32", 64, False) == 0


def test_append_of_many_sequences():
    """More sequences than one CTA has threads, most of them without new tokens."""
    rng = np.random.RandomState(0)
    counts = [int(rng.randint(1, 80)) if i % 7 == 0 else 0 for i in range(700)]
    lens = [c + int(rng.randint(0, 70)) for c in counts]
    assert _append_check("packed", counts, lens, 1, 1, 64, "bf16", 64, False) == 0
    # more than the kernel keeps the offsets of in shared memory
    counts = [int(rng.randint(1, 9)) if i % 5 == 0 else 0 for i in range(1500)]
    lens = [c + int(rng.randint(0, 70)) for c in counts]
    assert _append_check("packed", counts, lens, 1, 1, 64, "f32", 32, True) == 0


def test_append_skips_and_flags_bad_pages():
    def spoil(t):
        t[0, 1] = -1
        t[1, 0] = 1 << 30
    assert _append_check("packed", [100, 5], [130, 20], 2, 2, 64, "bf16", 64, False, spoil=spoil) == 5
    # more new tokens than the length holds: positions below zero
    dev = "cuda"
    call = hils.Append(1, 1, 1, 64, 1, "f32", inv_freq=_freq(64))
    kp = torch.zeros(1, 1, 64, 64, device=dev)
    k = torch.ones(4, 1, 64, device=dev)
    q_out = torch.full((4, 1, 64), 7.0, device=dev)
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device=dev)
    full = torch.empty(1, dtype=torch.int32, device=dev)
    call(k, k, kp, kp.clone(), i(0).view(1, 1), i(1), q=k, q_out=q_out, cu_new=i(0, 4), full_pages=full)
    assert call.device_status() == 5 and call.device_status() == 0
    assert (q_out[:3] == 7).all() and torch.equal(q_out[3], k[3]) and kp[0, 0, 1:].abs().max() == 0
    assert torch.equal(kp[0, 0, 0], k[0, 0]) and full.item() == -1
    # beyond the table: queries are rotated, nothing is written
    kp.zero_()
    call(k, k, kp, kp.clone(), i(0).view(1, 1), i(66), q=k, q_out=q_out, cu_new=i(0, 4))
    assert call.device_status() == 5
    want = CO.rotate(np.ones((1, 1, 4, 64)), _np(_freq(64)), [62, 63, 64, 65])[0, 0]
    _close(q_out[:, 0], want, 2.0 ** -18, "q")
    assert kp[0, 0, :62].abs().max() == 0 and kp[0, 0, 62:].abs().min() > 0


# ---- dense decode -----------------------------------------------------------
def _dense_case(lens, h, g, d, dtype, window=0, scale=None, seed=0, needles=True, garbage=False, spare=2):
    dt = DT[dtype]
    b = len(lens)
    max_chunks = max(1, -(-max(lens) // 64))
    pool = sum(-(-max(n, 0) // 64) for n in lens) + spare
    table = _table([max(n, 0) for n in lens], max_chunks, pool, seed)
    q = _randn(b, h, d, dtype=dt, seed=seed)
    kp, vp = _randn(pool, g, 64, d, dtype=dt, seed=seed + 1), _randn(pool, g, 64, d, dtype=dt, seed=seed + 2)
    if needles:
        for bi, n in enumerate(lens):
            if n > 0:
                j = (n * 7) // 11
                kp[table[bi, j // 64], :, j % 64] = (8 * q[bi, 0].float() / q[bi, 0].float().norm()).to(dt)
    if garbage:  # what lies behind the last token of each sequence, and in pages of none
        used = np.zeros((pool, 64), bool)
        for bi, n in enumerate(lens):
            for j in range(n):
                used[table[bi, j // 64], j % 64] = True
        free = torch.from_numpy(~used).cuda()
        for x, bad in ((kp, math.nan), (vp, math.inf)):
            x.transpose(1, 2)[free] = bad
    return dict(q=q, k_pages=kp, v_pages=vp, block_table=torch.from_numpy(table).cuda(),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device="cuda")), (window, scale)


def _dense_want(t, window, scale):
    d = t["q"].shape[-1]
    return CO.decode_dense(_np(t["q"]), _np(t["k_pages"]), _np(t["v_pages"]), t["block_table"].cpu().numpy(),
                           t["seq_lens"].cpu().numpy(), scale if scale is not None else d ** -0.5, window)


def _dense_close(out, lse, t, window, scale):
    want, wlse, mag, size = _dense_want(t, window, scale)
    d, n = t["q"].shape[-1], max(1, int(t["seq_lens"].max()))
    r = 2 * d * 2.0 ** -23 * size + 2.0 ** -16 + n * 2.0 ** -23
    _close(out, want, r[..., None] * mag + _u(out.dtype) * (np.abs(want) + r[..., None] * mag), "out")
    _close(lse, wlse, r + 2.0 ** -22 * np.abs(np.where(np.isfinite(wlse), wlse, 0)), "lse")


def _dense_run(t, window=0, scale=None):
    b, h, d = t["q"].shape
    call = hils.DenseDecode(b, h, t["k_pages"].shape[1], d, t["block_table"].shape[1], t["q"].dtype, window=window,
                            scale=scale)
    lse = torch.full((b, h), 5.0, device="cuda")
    out = call(**t, lse=lse)
    assert call.device_status() == 0
    return out, lse


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,g", [(2, 2), (4, 2), (8, 2), (16, 2), (8, 1)])
def test_dense_matches_oracle(dtype, d, h, g):
    t, w = _dense_case([1, 0, 64, 65, 1000, 63, 127, 16, 17, 33], h, g, d, dtype, seed=h + d, garbage=False)
    _dense_close(*_dense_run(t), t, *w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens,h,g,d", [([4500], 4, 1, 64), ([1], 1, 1, 64), ([0], 8, 1, 128), ([3001, 2], 2, 2, 128)])
def test_dense_few_sequences(dtype, lens, h, g, d):
    t, w = _dense_case(lens, h, g, d, dtype, seed=3)
    _dense_close(*_dense_run(t), t, *w)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [64, 128, 512])
def test_dense_window(dtype, window):
    t, _ = _dense_case([1, 64, 65, 700, 0, 512, 513, 129], 4, 2, 64, dtype, seed=window)
    _dense_close(*_dense_run(t, window=window), t, window, None)


@pytest.mark.parametrize("scale", [0.5, -0.25, 3.0])
def test_dense_scale(scale):
    t, _ = _dense_case([300, 31], 4, 2, 64, "f32", seed=9)
    _dense_close(*_dense_run(t, scale=scale), t, 0, scale)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lens", [[5, 64, 0, 193, 1], [2000]])
def test_dense_looks_at_nothing_behind_the_last_token(dtype, lens):
    t, w = _dense_case(lens, 8, 2, 64, dtype, seed=5, garbage=True)
    clean = {k: v.clone() for k, v in t.items()}
    for x in (clean["k_pages"], clean["v_pages"]):
        x.nan_to_num_(0.0, 0.0, 0.0)
    out, lse = _dense_run(t)
    _dense_close(out, lse, clean, *w)


def test_dense_infinite_and_missing_logits():
    """A key of -inf gets no weight; a row whose every logit is -inf is zero; NaN stays NaN."""
    for dtype in ("bf16", "f32"):
        t, w = _dense_case([200, 200, 200, 90], 2, 2, 64, dtype, seed=6, needles=False)
        t["q"] = t["q"].abs() + 0.5
        kp, vp, bt = t["k_pages"], t["v_pages"], t["block_table"].cpu().numpy()
        kp[bt[0, 1], :, 5] = -math.inf          # one key
        for c in range(4):
            kp[bt[1, c]] = -math.inf            # every key of sequence 1
        kp[bt[2, 0], :, 3] = math.nan
        kp[bt[3, 0]] = -math.inf                # a whole page, the rest is fine
        out, lse = _dense_run(t)
        assert torch.isfinite(out[0]).all() and (out[1] == 0).all() and torch.isnan(out[2]).all()
        assert (lse[1] == -math.inf).all()
        kk = _np(kp)
        ref = {**t, "k_pages": torch.from_numpy(np.where(np.isneginf(kk), -1e6, np.nan_to_num(kk, neginf=-1e6)))}
        want, wlse, mag, _ = _dense_want({**ref, "k_pages": ref["k_pages"].cuda()}, *w)
        for bi in (0, 3):
            r = 2 * 64 * 2.0 ** -23 * 200 + 2.0 ** -15
            _close(out[bi], want[bi], r * mag[bi] + 1.01 * _u(out.dtype) * np.abs(want[bi]) + 1e-9, "out")


def _dense_close_gpu(out, lse, t, lens, window=0):
    """The same bounds against the definition in 64 bits on the GPU, for long caches.  Their sums
    run over at most a few thousand terms at a time (units, warps, SMs): n = 4096."""
    b, h, d = t["q"].shape
    g = t["k_pages"].shape[1]
    want, wlse = torch.zeros(b, h, d).double(), torch.full((b, h), -math.inf).double()
    mag, size = torch.zeros(b, h, d).double(), torch.zeros(b, h).double()
    for bi, n in enumerate(lens):
        if n == 0:
            continue
        lo = max(0, ((n - 1) // 64 + 1 - window // 64) * 64) if window else 0
        pages = t["block_table"][bi, lo // 64:-(-n // 64)].long()
        for gi in range(g):
            k, v = (t[x][pages, gi].reshape(-1, d)[:n - lo].double() for x in ("k_pages", "v_pages"))
            rows = slice(gi * (h // g), (gi + 1) * (h // g))
            q = t["q"][bi, rows].double()
            s = q @ k.T * d ** -0.5
            p = torch.softmax(s, -1)
            wlse[bi, rows], want[bi, rows], mag[bi, rows] = torch.logsumexp(s, -1).cpu(), (p @ v).cpu(), (p @ v.abs()).cpu()
            size[bi, rows] = ((q.abs() @ k.abs().T).amax(-1) * d ** -0.5).cpu()
    want, wlse, mag, size = (x.numpy() for x in (want, wlse, mag, size))
    r = 2 * d * 2.0 ** -23 * size + 2.0 ** -16 + 4096 * 2.0 ** -23
    _close(out, want, r[..., None] * mag + _u(out.dtype) * (np.abs(want) + r[..., None] * mag), "out")
    _close(lse, wlse, r + 2.0 ** -22 * np.abs(np.where(np.isfinite(wlse), wlse, 0)), "lse")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("h,g,lens", [
    (2, 2, [60001, 333, 0, 20000, 7777]), (4, 2, [60001, 333, 0, 20000, 7777]), (8, 2, [60001, 333, 0, 20000, 7777]),
    (16, 2, [60001, 333, 0, 20000, 7777]),
    (8, 1, [150001]), (1, 1, [150001]), (2, 1, [99, 130000, 64]),  # one head cut between more than 32 SMs
])
def test_dense_long_caches(dtype, d, h, g, lens):
    """Enough keys that every stage of each SM's rings is filled several times, cut at odd
    places; the same bits each time."""
    t, _ = _dense_case(lens, h, g, d, dtype, seed=h + d)
    out, lse = _dense_run(t)
    for _ in range(3):
        again, again_lse = _dense_run(t)
        assert torch.equal(again, out) and torch.equal(again_lse, lse)
    _dense_close_gpu(out, lse, t, lens)


@pytest.mark.parametrize("b,h,g,d,most,window", [(70, 8, 2, 128, 700, 0), (300, 4, 4, 64, 300, 0),
                                                 (1100, 2, 1, 64, 200, 0), (90, 16, 2, 64, 3000, 256)])
def test_dense_batches_of_short_sequences(b, h, g, d, most, window):
    """Many (sequence, KV head)s per warp; more sequences than one launch takes."""
    rng = np.random.RandomState(b)
    lens = [0 if i % 11 == 3 else int(rng.randint(1, most)) for i in range(b)]
    for dtype in ("bf16", "f32"):
        t, _ = _dense_case(lens, h, g, d, dtype, seed=b, needles=False)
        out, lse = _dense_run(t, window=window)
        _dense_close_gpu(out, lse, t, lens, window)


def test_dense_with_tables_far_wider_than_the_lengths():
    """Tables of 67M tokens a sequence: one launch counts the units of 63 of them in 32 bits."""
    b, h, g, d = 70, 8, 8, 64
    t, w = _dense_case([int(x) for x in np.random.RandomState(1).randint(0, 200, b)], h, g, d, "bf16", seed=30)
    wide = torch.full((b, 1 << 20), -1, dtype=torch.int32, device="cuda")
    wide[:, :t["block_table"].shape[1]] = t["block_table"]
    out, lse = _dense_run(t)
    o, l = _dense_run({**t, "block_table": wide})
    _dense_close_gpu(o, l, t, t["seq_lens"].tolist())
    _dense_close_gpu(out, lse, t, t["seq_lens"].tolist())


def test_calls_on_a_given_stream_with_a_callers_workspace():
    t, w = _dense_case([700, 90], 4, 2, 64, "bf16", seed=31)
    want = _dense_run(t)[0]
    m = t["block_table"].shape[1]
    from chunk_wise_hierarchical_b200._abi import make_shape, workspace_size
    n = workspace_size(make_shape(2, 4, 2, 64, m * 64, 0, 1), hils.OP_DECODE_DENSE)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    call = hils.DenseDecode(2, 4, 2, 64, m, torch.bfloat16, ws=ws)
    q4 = _randn(2, 4, 70, 64, dtype=torch.bfloat16, seed=32)
    turned = hils.rotate(q4, _freq(64))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        out = call(**t, stream=side)
        r = hils.rotate(q4, _freq(64), stream=side)
        assert call.device_status(stream=side) == 0  # waits for the stream
        assert torch.equal(out, want) and torch.equal(r, turned)
    with pytest.raises(hils.HilsError):  # a workspace off its alignment is refused
        hils.DenseDecode(2, 4, 2, 64, m, torch.bfloat16, ws=torch.zeros(n + 8, dtype=torch.uint8, device="cuda")[8:])(**t)


def test_dense_every_length_of_a_ragged_batch():
    lens = list(range(0, 260)) + [1500, 3]
    t, w = _dense_case(lens, 2, 1, 64, "bf16", seed=11)
    _dense_close(*_dense_run(t), t, *w)


def test_dense_shared_pages_and_the_same_sequence_twice():
    t, w = _dense_case([640, 640, 100], 4, 2, 64, "bf16", seed=12)
    t["block_table"][1] = t["block_table"][0]
    t["q"][1] = t["q"][0]
    out, lse = _dense_run(t)
    _dense_close(out, lse, t, *w)


def test_dense_skips_and_flags_bad_pages():
    t, w = _dense_case([300, 300, 64], 4, 2, 64, "bf16", seed=13, needles=False)
    t["block_table"][0, 2] = -1
    t["block_table"][1, 0] = 1 << 30
    t["block_table"][2, 0] = t["k_pages"].shape[0]
    b, h, d = t["q"].shape
    call = hils.DenseDecode(b, h, 2, d, t["block_table"].shape[1], t["q"].dtype)
    lse = torch.empty(b, h, device="cuda")
    out = call(**t, lse=lse)
    assert call.device_status() == 5 and call.device_status() == 0
    _dense_close(out, lse, t, *w)
    assert (out[2] == 0).all()
    # a length beyond the table: its keys are those the table has
    t, w = _dense_case([300, 200], 4, 2, 64, "f32", seed=14)
    t["seq_lens"][0] = 64 * t["block_table"].shape[1] + 7
    call = hils.DenseDecode(2, 4, 2, 64, t["block_table"].shape[1], "f32")
    out = call(**t)
    assert call.device_status() == 5
    t["seq_lens"][0] = 64 * t["block_table"].shape[1]
    want = _dense_want(t, *w)[0]
    assert np.abs(_np(out) - want).max() < 1e-4


def test_dense_pool_beyond_32_bit_offsets():
    """Pages whose element offsets pass 2^31 and 2^32."""
    g, d, P = 8, 128, 68000  # 64 * 8 * 128 * 68000 = 4.46e9 elements, 8.9 GB each
    kp = torch.empty(P, g, 64, d, dtype=torch.bfloat16, device="cuda")
    vp = torch.empty_like(kp)
    ids = [0, 33000, P - 1, 65537]
    for n, p in enumerate(ids):
        kp[p] = _randn(g, 64, d, dtype=torch.bfloat16, seed=n)
        vp[p] = _randn(g, 64, d, dtype=torch.bfloat16, seed=n + 50)
    q = _randn(1, g, d, dtype=torch.bfloat16, seed=99)
    i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    # append the last 3 tokens there too
    k, v = _randn(3, g, d, dtype=torch.bfloat16, seed=100), _randn(3, g, d, dtype=torch.bfloat16, seed=101)
    hils.append_paged(k, v, kp, vp, i([ids]), i([250]), cu_new=i([0, 3]))
    out, lse = hils.decode_dense(q, kp, vp, i([ids]), i([250]), return_lse=True)
    small = dict(q=q, k_pages=kp[ids].clone(), v_pages=vp[ids].clone(), block_table=i([[0, 1, 2, 3]]), seq_lens=i([250]))
    assert torch.equal(small["k_pages"][3, :, 55:58], k.transpose(0, 1))
    _dense_close(out, lse, small, 0, None)


def test_dense_lse_joins_windows():
    """Two windows' outputs joined by their log masses give the whole."""
    t, w = _dense_case([640], 4, 2, 64, "f32", seed=15)
    out, lse = _dense_run(t)
    a, la = _dense_run(t, window=128)
    first = {**t, "seq_lens": t["seq_lens"] - 128}
    c, lc = _dense_run(first)
    z = torch.logaddexp(la, lc)
    joined = a * (la - z).exp()[..., None] + c * (lc - z).exp()[..., None]
    assert (z - lse).abs().max() < 2e-5 and (joined - out).abs().max() < 2e-5


# ---- streams, graphs, repeats -----------------------------------------------
def test_dense_repeats_bit_for_bit_and_on_another_stream():
    t, w = _dense_case([5000, 0, 700, 33, 2500], 8, 2, 128, "bf16", seed=16)
    out, lse = _dense_run(t)
    for _ in range(5):
        o, l = _dense_run(t)
        assert torch.equal(o, out) and torch.equal(l, lse)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    o, l = hils.decode_dense(**t, return_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(o, out) and torch.equal(l, lse)
    with torch.cuda.stream(side):
        call = hils.DenseDecode(5, 8, 2, 128, t["block_table"].shape[1], torch.bfloat16)
    torch.cuda.synchronize()
    assert torch.equal(call(**t), out)


def test_two_graphs_that_share_a_workspace():
    """One after the other on one stream, in any order, each keeps its own result."""
    t, _ = _dense_case([3000, 700, 0], 8, 2, 128, "bf16", seed=20)
    u, _ = _dense_case([900, 2800, 64], 8, 2, 128, "bf16", seed=21)
    m = t["block_table"].shape[1]
    u["block_table"] = torch.nn.functional.pad(u["block_table"], (0, m - u["block_table"].shape[1]), value=-1)
    call = hils.DenseDecode(3, 8, 2, 128, m, torch.bfloat16)
    want = [call(**x).clone() for x in (t, u)]
    graphs, outs = [], []
    for x in (t, u):
        out = torch.empty_like(x["q"])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(**x, out=out)
        graphs.append(g)
        outs.append(out)
    for i in (0, 1, 1, 0, 1, 0):
        outs[i].fill_(9)
        graphs[i].replay()
        assert torch.equal(outs[i], want[i])
    assert call.device_status() == 0


def test_captured_after_copies_and_a_join_of_streams():
    """The calls in a graph behind a copy, a memset and a join of two streams, each of which they
    have to wait for."""
    t, _ = _dense_case([2000, 700, 0], 8, 2, 64, "bf16", seed=22)
    call = hils.DenseDecode(3, 8, 2, 64, t["block_table"].shape[1], torch.bfloat16)
    f = _freq(64)
    src = [_randn(3, 8, 1, 64, dtype=torch.bfloat16, seed=s) for s in (40, 41, 42)]
    x, y = torch.empty_like(src[0]), torch.empty_like(src[0])
    pos = torch.tensor([[1999], [699], [0]], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    q, out, once = torch.empty_like(t["q"]), torch.empty_like(t["q"]), None
    big = torch.randn(1 << 24, device="cuda")

    def step():
        x.copy_(y)                                        # a copy
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z = (big * 2).sin_().sum() * 0                # long enough to be overtaken
            pos.add_(z.int())
        main.wait_stream(side)
        hils.rotate(x, f, positions=pos, q_out=q.view(3, 8, 1, 64))   # behind the join
        call(**{**t, "q": q}, out=out)
        return hils.decode_dense(**{**t, "q": out})       # its own workspace, cleared in the graph

    y.copy_(src[0])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once = step()
    for s in src[1:] + src[:1]:
        y.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        qs = hils.rotate(s, f, positions=pos)
        assert torch.equal(q, qs[:, :, 0])
        first = _dense_run({**t, "q": q})[0]
        assert torch.equal(out, first)
        assert torch.equal(once, _dense_run({**t, "q": out})[0])


def test_two_workspaces_at_once():
    t, _ = _dense_case([3000, 700], 8, 2, 64, "bf16", seed=17)
    u, _ = _dense_case([900, 2800], 8, 2, 64, "bf16", seed=18)
    want = [_dense_run(x)[0] for x in (t, u)]
    calls = [hils.DenseDecode(2, 8, 2, 64, x["block_table"].shape[1], torch.bfloat16) for x in (t, u)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for c, s, x, o in zip(calls, streams, (t, u), outs):
            with torch.cuda.stream(s):
                o.append(c(**x))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(w, y) for y in o)


def test_a_decode_step_in_a_graph():
    """rotate + append + summaries of the filled pages + both decodes, captured once and
    replayed while the lengths grow on the device: each step against a fresh eager call."""
    b, h, g, d, K = 2, 4, 2, 64, 3
    dt = torch.bfloat16
    max_chunks, pool = 5, 12
    table = torch.from_numpy(_table([320, 320], max_chunks, pool, 3)).cuda()
    kp, vp = torch.zeros(pool, g, 64, d, dtype=dt, device="cuda"), torch.zeros(pool, g, 64, d, dtype=dt, device="cuda")
    lm = _randn(pool, h, d, dtype=dt, seed=1)
    kbar, hb = torch.zeros(pool, h, d, device="cuda"), torch.zeros(pool, h, device="cuda")
    lens = torch.tensor([60, 190], dtype=torch.int32, device="cuda")
    f = _freq(64)
    fused = torch.empty(b, h + 2 * g, d, dtype=dt, device="cuda")
    app = hils.Append(b, h, g, d, max_chunks, dt, inv_freq=f)
    dense = hils.DenseDecode(b, h, g, d, max_chunks, dt)
    sparse = hils.Decode(b, h, g, d, max_chunks, K, dt)
    q = torch.empty(b, h, d, dtype=dt, device="cuda")
    full = torch.empty(hils.append_slots(b, b), dtype=torch.int32, device="cuda")
    out_d, out_s, lse = torch.empty_like(q), torch.empty_like(q), torch.empty(b, h, device="cuda")
    # the prompts
    n0 = lens.tolist()
    prompt = _randn(sum(n0), h + 2 * g, d, dtype=dt, seed=2)
    cu = torch.tensor([0, n0[0], sum(n0)], dtype=torch.int32, device="cuda")
    pf = torch.empty(hils.append_slots(b, sum(n0)), dtype=torch.int32, device="cuda")
    app(prompt[:, h:h + g], prompt[:, h + g:], kp, vp, table, lens, cu_new=cu, full_pages=pf)
    hils.summarize_paged(kp, lm, pf, kbar, hb)

    def step():
        lens.add_(1)
        app(fused[:, h:h + g], fused[:, h + g:], kp, vp, table, lens, q=fused[:, :h], q_out=q, full_pages=full)
        hils.summarize_paged(kp, lm, full, kbar, hb)
        dense(q, kp, vp, table, lens, out=out_d, lse=lse)
        sparse(q, kp, vp, kbar, hb, table, lens, out=out_s)

    state = [x.clone() for x in (lens, kp, vp, kbar, hb)]
    fused.copy_(_randn(b, h + 2 * g, d, dtype=dt, seed=99))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for x, y in zip((lens, kp, vp, kbar, hb), state):
        x.copy_(y)
    rows = [[prompt[:n0[0], h:]], [prompt[n0[0]:, h:]]]
    for i in range(8):  # sequence 0 fills its first page at the fourth step, sequence 1 at the second
        new = _randn(b, h + 2 * g, d, dtype=dt, seed=10 + i)
        fused.copy_(new)
        for bi in range(b):
            rows[bi].append(new[bi:bi + 1, h:])
        graph.replay()
        torch.cuda.synchronize()
        n = [x + i + 1 for x in n0]
        assert lens.tolist() == n and app.device_status() == 0 and dense.device_status() == 0
        want = hils.rotate(new[:, None, :h].transpose(1, 2), f,
                           positions=torch.tensor([[x - 1] for x in n], dtype=torch.int32, device="cuda"))
        assert torch.equal(q, want[:, :, 0])
        _dense_close(out_d, lse, dict(q=q, k_pages=kp, v_pages=vp, block_table=table, seq_lens=lens), 0, None)
        for bi in range(b):
            # the pages hold the rotated rows, as rotating the whole sequence gives them
            kv = torch.cat(rows[bi])
            kr = hils.rotate(kv[None, :, :g].transpose(1, 2).contiguous(), f)[0]
            for c in range(-(-n[bi] // 64)):
                m = min(64, n[bi] - 64 * c)
                p = int(table[bi, c])
                assert torch.equal(kp[p, :, :m], kr[:, 64 * c:64 * c + m])
                assert torch.equal(vp[p, :, :m].transpose(0, 1), kv[64 * c:64 * c + m, g:])
        ref = O.decode(q.cpu(), kp.cpu(), vp.cpu(), lm.cpu(), table.cpu().numpy(), lens.cpu().numpy(), K)
        check_close(out_s.float().cpu().numpy(), ref["out"], True)


def test_prompt_through_the_framework():
    """A prompt as a user runs it: rotated projections through attend, the same tokens appended
    to the cache; the last row from the cache (K = all chunks, so both layers see every key)."""
    b, h, g, n, d = 2, 4, 2, 190, 64
    dt = torch.bfloat16
    fused = _randn(b, n, h + 2 * g, d, dtype=dt, seed=30)
    f = _freq(d)
    sl = [fused[:, :, i:j].transpose(1, 2) for i, j in ((0, h), (h, h + g), (h + g, h + 2 * g))]
    q, k = hils.rotate(sl[0], f, k=sl[1])
    v = sl[2].contiguous()
    lm = _randn(b, h, n // 64, d, dtype=dt, seed=31)
    out, lse = hils.attend(q, k, v, lm, 4, return_lse=True)
    table = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    kp, vp = torch.zeros(6, g, 64, d, dtype=dt, device="cuda"), torch.zeros(6, g, 64, d, dtype=dt, device="cuda")
    lens = torch.full((b,), n, dtype=torch.int32, device="cuda")
    full = torch.empty(hils.append_slots(b, b * n), dtype=torch.int32, device="cuda")
    qa = hils.append_paged(sl[1], sl[2], kp, vp, table, lens, inv_freq=f, q=sl[0], full_pages=full)
    assert torch.equal(qa, q)
    assert sorted(x for x in full.tolist() if x >= 0) == [0, 1, 3, 4]
    flat = kp.view(2, 3, g, 64, d).transpose(1, 2).reshape(b, g, 192, d)[:, :, :n]
    assert torch.equal(flat, k)
    lp = torch.zeros(6, h, d, dtype=dt, device="cuda")
    lp.view(2, 3, h, d)[:, :2] = lm.transpose(1, 2)
    kbar, hb = torch.zeros(6, h, d, device="cuda"), torch.zeros(6, h, device="cuda")
    hils.summarize_paged(kp, lp, full, kbar, hb)
    last = q[:, :, -1].contiguous()
    sparse = hils.decode(last, kp, vp, kbar, hb, table, lens, 4)
    assert (sparse.float() - out[:, :, -1].float()).abs().max() < 2e-2
    dense, dl = hils.decode_dense(last, kp, vp, table, lens, return_lse=True)
    _dense_close(dense, dl, dict(q=last, k_pages=kp, v_pages=vp, block_table=table, seq_lens=lens), 0, None)


# ---- weights and values of the dense decode ---------------------------------
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,g,d", [(1, 1, 64), (4, 1, 128), (8, 1, 64)])
def test_dense_weights_keep_32_bits(dtype, h, g, d):
    """Values that cancel: what is left shows how exactly the weights entered.  Each query has one
    element, so a logit is one exact product times a scale of two roundings: |s log2 e| <= 2 gives
    3 * 2^-23 absolute, exp2f 2 steps of 2^-23: a weight is off by 2^-21, and so is their sum; fp32
    sums of 6 terms in three parts by 18 * 2^-24.  r = 2^-19 of sum p |v| holds all of them; two
    bf16 parts (2^-17 each) do not fit."""
    b, n = 48, 6
    dt = DT[dtype]
    rng = np.random.RandomState(d + h)
    logit = torch.from_numpy(rng.uniform(0, 1.3, (b, n))).to(dt)
    q = torch.zeros(b, h, d, dtype=dt)
    q[:, :, 5] = 1
    kp, vp = torch.zeros(b, g, 64, d, dtype=dt), torch.zeros(b, g, 64, d, dtype=dt)
    kp[:, 0, :n, 5] = logit
    p = np.exp(_np(logit))
    p /= p.sum(-1, keepdims=True)
    v = np.zeros((b, n, d))
    v[:, 0] = _np(torch.from_numpy(rng.uniform(1, 2, (b, d))).to(dt))
    for j in range(1, n):
        left = (p[:, :j, None] * v[:, :j]).sum(1)
        v[:, j] = _np(torch.from_numpy(-left / p[:, j, None]).to(dt))
    vp[:, 0, :n] = torch.from_numpy(v).to(dt)
    t = dict(q=q.cuda(), k_pages=kp.cuda(), v_pages=vp.cuda(),
             block_table=torch.arange(b, dtype=torch.int32, device="cuda").view(b, 1),
             seq_lens=torch.full((b,), n, dtype=torch.int32, device="cuda"))
    out, _ = _dense_run(t, scale=1.0)
    want = (p[..., None] * v).sum(1)[:, None].repeat(h, 1)
    mag = (p[..., None] * np.abs(v)).sum(1)[:, None].repeat(h, 1)
    assert np.abs(want).max() < 2.0 ** -20
    _close(out, want, 2.0 ** -19 * mag + _u(dt) * (np.abs(want) + 2.0 ** -19 * mag), "out")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("h,g,d", [(2, 2, 64), (16, 2, 128)])
def test_dense_infinite_values(dtype, h, g, d):
    """A value times its weight, as the formula has it: an infinity wherever the weight is not
    zero, NaN where both infinities meet or one meets a weight of zero; other columns are as they
    were."""
    lens = [200, 90, 1, 3000, 70]
    t, w = _dense_case(lens, h, g, d, dtype, seed=60, needles=False)
    vp, kp, bt = t["v_pages"], t["k_pages"], t["block_table"].cpu().numpy()
    clean = {k: v.clone() for k, v in t.items()}
    put = lambda bi, j, col, x: vp[bt[bi, j // 64], :, j % 64].__setitem__((slice(None), col), x)
    for j in range(0, 200, 7):
        put(0, j, j % d, math.inf)
    put(1, 3, 9, -math.inf)
    put(1, 80, 9, math.inf)
    put(1, 81, 10, math.inf)
    put(2, 0, 4, -math.inf)         # a weight of one
    put(3, 1777, 11, -math.inf)     # in a partial
    kp[bt[4, 0], :, 20] = -math.inf * torch.sign(t["q"][4, :: h // g]).to(kp.dtype)  # head 0 of each group: no weight
    put(4, 20, 12, math.inf)
    out, lse = _dense_run(t)
    want, wlse, mag, size = _dense_want(clean, *w)
    spot = np.zeros(want.shape)
    for j in range(0, 200, 7):
        spot[0, :, j % d] = math.inf
    spot[1, :, 9], spot[1, :, 10], spot[2, :, 4], spot[3, :, 11] = math.nan, math.inf, -math.inf, -math.inf
    got = _np(out)
    assert np.isnan(got[4, ::h // g, 12]).all()
    some = spot != 0
    assert np.array_equal(got[some], spot[some], equal_nan=True)
    rest = ~some
    rest[4] = False
    r = (2 * d * 2.0 ** -23 * size + 2.0 ** -16 + 3000 * 2.0 ** -23)[..., None] * mag
    assert (np.abs(got - want)[rest] <= (r + _u(out.dtype) * (np.abs(want) + r))[rest]).all()


def test_dense_sums_of_a_long_run_are_rounded():
    """Values 1 and then -1 at the same keys: every weight is cancelled by its own likeness, and
    what is left is the error of the sums alone.  148 * 8 (sequence, KV head)s of 64 units: a
    warp's run is one of them.  A rounded sum of u units, at most half of M = sum p |v| on its
    way, is off by u 2^-25 M; a unit's own sum (four products of the leading parts, each cut off
    at 2^-23; the small parts' add less than one more) by 5 * 2^-23 of its share: 42 * 2^-24 M
    in all.  Cutting the running sum off at each of its 512 products loses about 92 * 2^-24 M."""
    b, g, d, n = 148, 8, 64, 64
    dt = torch.bfloat16
    q = _randn(b, g, d, dtype=dt, seed=70)
    half = _randn(n // 2, g, 64, d, dtype=dt, seed=71)
    kp = torch.cat((half, half))
    vp = torch.ones_like(kp)
    vp[n // 2:] = -1
    t = dict(q=q, k_pages=kp, v_pages=vp, seq_lens=torch.full((b,), 64 * n, dtype=torch.int32, device="cuda"),
             block_table=torch.arange(n, dtype=torch.int32, device="cuda").repeat(b, 1))
    out, _ = _dense_run(t)
    assert out.float().abs().max() <= 42 * 2.0 ** -24 * (1 + 2.0 ** -8)


# ---- rows between rows ------------------------------------------------------
def test_rotate_into_the_slices_of_a_fused_tensor():
    """backward's dq and dk rotated back to where the fused projection's gradient has them; the
    slice of v stays."""
    b, h, g, n, d = 2, 4, 4, 70, 64
    f = _freq(d)
    dq, dk = (_randn(b, x, n, d, dtype=torch.float32, seed=x + i) for i, x in ((80, h), (81, g)))
    for dt in (torch.float32, torch.bfloat16):
        want = hils.rotate(dq, f, k=dk, inverse=True, q_out=torch.empty_like(dq, dtype=dt), k_out=torch.empty_like(dk, dtype=dt))
        for shape, cut in (((b, n, h + 2 * g, d), lambda x, i: x[:, :, (0, h, h + g)[i]:][:, :, :h].transpose(1, 2)),
                           ((b, h + 2 * g, n, d), lambda x, i: x[:, (0, h, h + g)[i]:][:, :h]),
                           ((b, n, h, 3, d), lambda x, i: x[:, :, :, i].transpose(1, 2))):
            x = torch.full(shape, 7.0, dtype=dt, device="cuda")
            hils.rotate(dq, f, k=dk, inverse=True, q_out=cut(x, 0), k_out=cut(x, 1))
            assert torch.equal(cut(x, 0), want[0]) and torch.equal(cut(x, 1), want[1]) and (cut(x, 2) == 7).all()
            # and forward again, in place
            again = hils.rotate(*(y.clone() for y in want[:1]), f, k=want[1].clone())
            hils.rotate(cut(x, 0), f, k=cut(x, 1), q_out=cut(x, 0), k_out=cut(x, 1))
            assert torch.equal(cut(x, 0), again[0]) and torch.equal(cut(x, 1), again[1]) and (cut(x, 2) == 7).all()


def test_append_rotates_queries_in_the_fused_projection():
    b, h, g, d = 3, 4, 2, 64
    fused = _randn(b, h + 2 * g, d, dtype=torch.bfloat16, seed=83)
    ref = fused.clone()
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    f, lens, table = _freq(d), i(70, 1, 64), i(0, 1, 2, 3, 4, 5).view(3, 2)
    kp, vp = (torch.zeros(6, g, 64, d, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    kq, vq = kp.clone(), vp.clone()
    want = hils.append_paged(ref[:, h:h + g], ref[:, h + g:], kp, vp, table, lens, inv_freq=f, q=ref[:, :h])
    got = hils.append_paged(fused[:, h:h + g], fused[:, h + g:], kq, vq, table, lens, inv_freq=f, q=fused[:, :h],
                            q_out=fused[:, :h])
    assert torch.equal(got, want) and torch.equal(fused[:, h:], ref[:, h:])
    assert torch.equal(kp, kq) and torch.equal(vp, vq)


# ---- kernels that start while their predecessor runs ------------------------
def test_inputs_that_the_kernel_before_has_just_written():
    """A rotation writes the frequencies that the next rotation and append read, the append the
    queries that the dense decode reads: captured, and replayed with other values each time."""
    b, h, g, d = 4, 8, 2, 64
    i = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    t, _ = _dense_case([700, 129, 2000, 1], h, g, d, "bf16", seed=90)
    m = t["block_table"].shape[1]
    first = _freq(d)
    raw = torch.empty(1, 1, 1, d, device="cuda")               # its rotated row's head: the frequencies
    row, freq = torch.empty_like(raw), None
    freq = row.view(-1)[:d // 2]
    fused, q = torch.empty(b, h + 2 * g, d, dtype=torch.bfloat16, device="cuda"), torch.empty_like(t["q"])
    turned = torch.empty(1, h, b, d, dtype=torch.bfloat16, device="cuda")
    app = hils.Append(b, h, g, d, m, torch.bfloat16, inv_freq=freq)
    dense = hils.DenseDecode(b, h, g, d, m, torch.bfloat16)
    pos, out, n = i(3), torch.empty_like(q), t["seq_lens"]

    def step():
        for _ in range(3):
            hils.rotate(raw, first, positions=pos, q_out=row)
            hils.rotate(fused[None, :, :h].transpose(1, 2), freq, positions=n, q_out=turned)
            app(fused[:, h:h + g], fused[:, h + g:], t["k_pages"], t["v_pages"], t["block_table"], n, q=fused[:, :h], q_out=q)
            dense(q, t["k_pages"], t["v_pages"], t["block_table"], n, out=out)

    raw.fill_(0.1)
    fused.zero_()
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in range(4):
        raw.copy_(_randn(1, 1, 1, d, dtype=torch.float32, seed=91 + s))
        fused.copy_(_randn(b, h + 2 * g, d, dtype=torch.bfloat16, seed=95 + s))
        graph.replay()
        torch.cuda.synchronize()
        f = hils.rotate(raw, first, positions=pos).view(-1)[:d // 2].clone()
        torch.cuda.synchronize()
        assert torch.equal(f, freq)
        assert torch.equal(turned, hils.rotate(fused[None, :, :h].transpose(1, 2), f, positions=n))
        kp, vp = t["k_pages"].clone(), t["v_pages"].clone()
        torch.cuda.synchronize()
        qs = hils.append_paged(fused[:, h:h + g], fused[:, h + g:], kp, vp, t["block_table"], n, inv_freq=f, q=fused[:, :h])
        torch.cuda.synchronize()
        assert torch.equal(q, qs) and torch.equal(kp, t["k_pages"]) and torch.equal(vp, t["v_pages"])
        assert torch.equal(out, _dense_run({**t, "q": q.clone()})[0])


def test_captured_behind_writes_that_change_with_every_replay():
    """Positions written by a second stream that joins late, and a workspace whose counters another
    stream's call left dirty until a node of the graph clears it: a call that overtakes either
    shows."""
    t, _ = _dense_case([2000, 700, 0], 8, 2, 64, "bf16", seed=22)
    f = _freq(64)
    x = _randn(3, 8, 1, 64, dtype=torch.bfloat16, seed=40)
    pos, new_pos = (torch.zeros(3, 1, dtype=torch.int32, device="cuda") for _ in range(2))
    side = torch.cuda.Stream()
    q, out = torch.empty_like(t["q"]), torch.empty_like(t["q"])
    big = torch.randn(1 << 24, device="cuda")
    from chunk_wise_hierarchical_b200._abi import make_shape, workspace_size
    m = t["block_table"].shape[1]
    ws = torch.zeros(workspace_size(make_shape(3, 8, 2, 64, m * 64, 0, 1), hils.OP_DECODE_DENSE), dtype=torch.uint8, device="cuda")
    call = hils.DenseDecode(3, 8, 2, 64, m, torch.bfloat16, ws=ws)

    def step():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            z = (big * 2).sin_().sum() * 0                # long enough to be overtaken
            pos.copy_(new_pos + z.int())
            ws.zero_()
        main.wait_stream(side)
        hils.rotate(x, f, positions=pos, q_out=q.view(3, 8, 1, 64))
        call(**{**t, "q": q}, out=out)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for s in range(3):
        new_pos.copy_(torch.tensor([[1999 + s], [3 * s], [100 * s]], dtype=torch.int32))
        pos.fill_(-77)
        ws.fill_(1)  # counters that no join would find its last part by
        graph.replay()
        torch.cuda.synchronize()
        want = hils.rotate(x, f, positions=new_pos.clone())
        assert torch.equal(q, want[:, :, 0])
        assert torch.equal(out, _dense_run({**t, "q": q.clone()})[0]) and call.device_status() == 0


def test_rotate_angles_at_the_farthest_positions():
    """(1, 0) turned by p w, near the largest int32 p, against exact rationals: the remainder 2 t
    (half turns, at most 1) is rounded to fp32, pi 2^-25 of angle, and sincospif is good to 2 steps
    of 2^-24; 1 cos - 0 sin and 0 cos + 1 sin are exact."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    rng = np.random.RandomState(0)
    w = torch.from_numpy(rng.uniform(0.5, 1, 32).astype(np.float32))
    p = torch.from_numpy(2**31 - 1 - rng.randint(0, 1 << 20, 64)).int()
    p[::2] = -p[::2]
    x = torch.zeros(1, 1, 64, 64, device="cuda")
    x[..., :32] = 1
    got = _np(hils.rotate(x, w.cuda(), positions=p.cuda()))[0, 0]
    want = np.empty((64, 64))
    for i, a in enumerate(p.tolist()):
        for j, b in enumerate(w.tolist()):
            turns = Decimal(a) * Decimal(b) / (2 * pi)
            ang = float((turns - turns.to_integral_value()) * 2 * pi)
            want[i, j], want[i, 32 + j] = math.cos(ang), math.sin(ang)
    assert np.abs(got - want).max() <= math.pi * 2.0 ** -25 + 2.0 ** -23


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("window", [64 * 128, 64 * 129, 64 * 1000, 64 * ((1 << 25) - 1)])
def test_dense_wide_windows(dtype, window):
    lens = [64 * 129 + 5, 20000, 70001, 0, 64 * 130, 100]
    t, _ = _dense_case(lens, 4, 2, 64, dtype, seed=85)
    out, lse = _dense_run(t, window=window)
    _dense_close_gpu(out, lse, t, lens, window)


def test_append_for_no_sequences_lists_no_pages():
    call = hils.Append(0, 2, 2, 64, 3, torch.bfloat16)
    k = torch.zeros(130, 2, 64, dtype=torch.bfloat16, device="cuda")
    pages = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16, device="cuda")
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    full = torch.full((hils.append_slots(0, 130),), 99, dtype=torch.int32, device="cuda")
    call(k, k, pages, pages.clone(), i(0, 3), i(0), cu_new=i(1), full_pages=full)
    assert full.tolist() == [-1, -1]


@pytest.mark.parametrize("dtype,h,g", [("bf16", 8, 2), ("f32", 2, 2)])
def test_dense_in_place(dtype, h, g):
    """out may be q itself: cut between warps and SMs, whole, and empty."""
    t, _ = _dense_case([9000, 5, 0, 700, 64], h, g, 128, dtype, seed=86)
    want, lse = _dense_run(t)
    call = hils.DenseDecode(5, h, g, 128, t["block_table"].shape[1], t["q"].dtype)
    for _ in range(3):
        q, l = t["q"].clone(), torch.empty_like(lse)
        assert call(**{**t, "q": q}, out=q, lse=l) is q
        assert torch.equal(q, want) and torch.equal(l, lse)


@pytest.mark.parametrize("h,g,n", [(8, 1, 40), (32, 8, 40), (32, 8, 600), (32, 8, 5000), (24, 3, 6000), (9, 9, 5000)])
def test_rotate_blocks_of_heads(h, g, n):
    """However the heads are dealt to blocks, each is turned as it is alone."""
    f, dt = _freq(64), torch.bfloat16
    fused = _randn(1, n, h + 2 * g, 64, dtype=dt, seed=h + n)
    q, k = fused[:, :, :h].transpose(1, 2), fused[:, :, h:h + g].transpose(1, 2)
    qo, ko = hils.rotate(q, f, k=k)
    for x, y in ((q, qo), (k, ko)):
        for i in range(x.shape[1]):
            assert torch.equal(y[:, i:i + 1], hils.rotate(x[:, i:i + 1], f))
