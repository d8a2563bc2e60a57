"""The paged-cache operators on the host: their oracle against closed forms, the argument
checks of the binding (CPU tensors) and of the C ABI (nothing is launched)."""
import ctypes

import numpy as np
import pytest
import torch

import chunk_wise_hierarchical_b200 as hils
from chunk_wise_hierarchical_b200 import _abi
from chunk_wise_hierarchical_b200._abi import (HILS_BF16, HILS_F32, check_append_args, check_dense_args,
                                               check_rotate_args, make_shape)
from oracle import cache_oracle as CO
from oracle import hils_oracle as O

BF = torch.bfloat16
P_ = ctypes.c_void_p
FAKE = P_(1 << 20)  # never dereferenced


class Rows(ctypes.Structure):  # hils_rows
    _fields_ = [("data", P_), ("batch_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("token_stride", ctypes.c_int64)]


class Rope(ctypes.Structure):  # hils_rope
    _fields_ = [("inv_freq", P_), ("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32)]


# ---- the oracle -------------------------------------------------------------
def test_oracle_rotation_keeps_relative_positions():
    """q(p).k(r) depends on p - r alone, pairs keep their length, and the inverse undoes it."""
    rng = np.random.default_rng(0)
    f = 10000.0 ** (-np.arange(0, 32, 2) / 32)
    for inter in (False, True):
        q, k = rng.standard_normal((2, 64))
        dots = [CO.rotate_row(q, p + 7, f, inter) @ CO.rotate_row(k, p, f, inter) for p in (0, 1, 50, 4000)]
        assert np.allclose(dots, dots[0], atol=1e-9)
        assert np.isclose(np.linalg.norm(CO.rotate_row(q, 99, f, inter)), np.linalg.norm(q))
        assert np.allclose(CO.rotate_row(CO.rotate_row(q, 99, f, inter), 99, f, inter, inverse=True), q)
    assert np.allclose(CO.rotate_row([1.0] + [0.0] * 63, 1, [np.pi / 2], False)[:2], [0, 1])
    assert np.array_equal(CO.rotate_row(np.ones(64), 5, f)[32:], np.ones(32))


def test_oracle_dense_decode_is_the_last_row_of_dense_attention():
    """Against the prefill oracle with exact masses and every chunk (dense causal attention)."""
    rng = np.random.default_rng(1)
    n, d = 150, 64
    q, k, v = rng.standard_normal((3, n, d))
    t = lambda x: torch.from_numpy(x).view(1, 1, -1, d)
    ref = O.forward(t(q), t(k), t(v), torch.zeros(1, 1, n // 64, d, dtype=torch.float64), 64, 2, mode="exact")
    pages = np.zeros((4, 1, 64, d))
    vpages = np.zeros((4, 1, 64, d))
    for c, p in enumerate((2, 0, 3)):
        m = min(64, n - 64 * c)
        pages[p, 0, :m], vpages[p, 0, :m] = k[64 * c:64 * c + m], v[64 * c:64 * c + m]
    out, lse, _, _ = CO.decode_dense(q[-1].reshape(1, 1, d), pages, vpages, [[2, 0, 3]], [n], d ** -0.5)
    assert np.allclose(out[0, 0], ref["out"][0, 0, -1], atol=1e-12)
    assert np.isclose(lse[0, 0], ref["lse"][0, 0, -1])


# ---- the binding's checks ---------------------------------------------------
# On the host a call whose arguments are right goes as far as its launch, which then misses the
# GPU: "CUDA device".  A refusal says something else, and comes before.
def _right(call, *args, **kw):
    with pytest.raises(ValueError, match="CUDA device"):
        call(*args, **kw)


def _refused(call, *args, **kw):
    with pytest.raises((ValueError, TypeError)) as e:
        call(*args, **kw)
    assert "CUDA device" not in str(e.value)


def _ws(n=1 << 22):
    return torch.zeros(n, dtype=torch.uint8)


B, H, G, N, D = 2, 8, 2, 70, 64


def test_rotate_arguments():
    q, k = torch.zeros(B, H, N, D, dtype=BF), torch.zeros(B, G, N, D, dtype=BF)
    f = torch.ones(16)
    assert check_rotate_args(q, f, k) == 0
    assert check_rotate_args(q, f, k, torch.zeros(N, dtype=torch.int32)) == 0
    assert check_rotate_args(q, f, k, torch.zeros(B, N, dtype=torch.int32)) == N
    check_rotate_args(q, f, k, q_out=q, k_out=k)  # in place
    check_rotate_args(q, f, k, q_out=torch.zeros(B, H, N, D), k_out=torch.zeros(B, G, N, D))
    fused = torch.zeros(B, N, H + 2 * G, D, dtype=BF)
    check_rotate_args(fused[:, :, :H].transpose(1, 2), f, fused[:, :, H:H + G].transpose(1, 2))


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(B, G, N - 1, D, dtype=BF)),
    dict(k=torch.zeros(B, G, N, D)),
    dict(k=torch.zeros(G, N, D, dtype=BF)),
    dict(positions=torch.zeros(N, dtype=torch.int64)),
    dict(positions=torch.zeros(N + 1, dtype=torch.int32)),
    dict(positions=torch.zeros(1, N, dtype=torch.int32)),
    dict(positions=torch.zeros(2 * N, dtype=torch.int32)[::2]),
    dict(q_out=torch.zeros(B, H, N, D, dtype=torch.float16)),
    dict(q_out=torch.zeros(B, H, N + 1, D, dtype=BF)),
    dict(k_out=torch.zeros(B, G, N, D, dtype=BF)),
    dict(inv_freq=None),
])
def test_rotate_refuses(kw):
    a = dict(q=torch.zeros(B, H, N, D, dtype=BF), inv_freq=torch.ones(16))
    a.update(kw)
    with pytest.raises((ValueError, TypeError)):
        check_rotate_args(**a)
    _refused(hils.rotate, **a)
    if "k" not in kw and "k_out" not in kw:
        _refused(hils.rotate, k=torch.zeros(B, G, N, D, dtype=BF), **a)


def test_rotate_takes_what_is_right_as_far_as_the_device():
    q, k, f = torch.zeros(B, H, N, D, dtype=BF), torch.zeros(B, G, N, D, dtype=BF), torch.ones(16)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for kw in (dict(), dict(k=k), dict(k=k, positions=i(B, N)), dict(k=k, positions=i(N)), dict(k=k, q_out=q, k_out=k),
               dict(k=k, q_out=q.float(), k_out=k.float()), dict(k=k, k_out=k.clone())):
        _right(hils.rotate, q, f, **kw)


def test_rotate_refuses_overlapping_and_expanded_outputs():
    """By hils_rotate, before anything is launched: addresses are compared, not read."""
    L, ref = hils.lib(), ctypes.byref
    s, ro = _sh(seq_len=70), Rope(1 << 20, 32, 0)  # q [2, 8, 70, 64], k [2, 2, 70, 64] bf16
    base, qn = 1 << 20, 2 * 8 * 70 * 64
    dense = lambda p, h: Rows(p, h * 70 * 64, 70 * 64, 64)
    q, k = dense(base, 8), dense(base + (1 << 24), 2)
    qo, ko = dense(base + (2 << 24), 8), dense(base + (3 << 24), 2)

    def call(q=q, k=k, qo=qo, ko=ko, od=1):
        return L.hils_rotate(ref(s), ref(q), ref(k), ref(ro), None, 0, 0, ref(qo), ref(ko), od, None)

    assert call(qo=dense(base + 128, 8)) == 1                     # shifted by one row
    assert call(qo=dense(base + 2 * qn - 16, 8)) == 1             # its end
    assert call(qo=dense(k.data, 8)) == 1                         # on the other input
    assert call(ko=dense(qo.data, 2)) == 1                        # on the other output
    assert call(ko=dense(base, 2)) == 1                           # k_out on q
    assert call(qo=q, od=0) == 1                                  # in place with another type
    expanded = Rows(base, 70 * 64, 0, 64)
    assert call(q=expanded, qo=expanded) == 1                     # one memory for every head, in place
    assert call(qo=Rows(qo.data, 8 * 70 * 64, 70 * 64, 56)) == 1  # rows that share elements
    assert call(qo=Rows(qo.data, 0, 70 * 64, 64)) == 1
    assert call(q=Rows(base, -64, 70 * 64, 64)) == 1


@pytest.mark.parametrize("f", [torch.ones(0), torch.ones(4), torch.ones(40), torch.ones(16, dtype=torch.float64),
                               torch.ones(4, 4), torch.ones(32)[::2]])
def test_rope_refuses(f):
    with pytest.raises((ValueError, TypeError)):
        _abi._rope_bytes(f, False, 64)


def test_structs_are_packed_as_declared():
    t = torch.zeros(2, 3, 5, 64, dtype=BF)
    r = Rows.from_buffer_copy(_abi._rows4(t))
    assert (r.data, r.batch_stride, r.head_stride, r.token_stride) == (t.data_ptr(), 960, 320, 64)
    r = Rows.from_buffer_copy(_abi._rows_packed(t[0]))
    assert (r.head_stride, r.token_stride) == (64, 320)
    r = Rows.from_buffer_copy(_abi._rows_single(t[0]))
    assert (r.batch_stride, r.head_stride, r.token_stride) == (320, 64, 0)
    f = torch.ones(24)
    o = Rope.from_buffer_copy(_abi._rope_bytes(f, True, 64))
    assert (o.inv_freq, o.rotary_dim, o.interleaved) == (f.data_ptr(), 48, 1)


def test_tensors_that_are_not_contiguous_are_refused():
    x = torch.zeros(2, 3, 64, 8, dtype=BF).transpose(2, 3)  # rows of stride 8
    y = torch.zeros(2, 3, 8, 64, dtype=BF)
    _refused(hils.rotate, x, torch.ones(16))
    _refused(hils.rotate, y, torch.ones(16), q_out=x)
    _refused(hils.rotate, y, torch.ones(16), k=x)
    call = hils.Append(B, H, G, D, 3, BF, ws=_ws())
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    for kw in (dict(k=torch.zeros(9, D, G, dtype=BF).transpose(1, 2)), dict(q=torch.zeros(9, D, H, dtype=BF).transpose(1, 2)),
               dict(k_pages=torch.zeros(5, 64, G, D, dtype=BF).transpose(1, 2)), dict(block_table=i(3, B).T),
               dict(seq_lens=i(2 * B)[::2]), dict(cu_new=i(2 * B + 2)[::2]), dict(full_pages=i(2 * B)[::2])):
        a = _append_args(**kw)
        a.pop("max_chunks")
        _refused(call, **a)
    call = hils.DenseDecode(B, H, G, D, 3, BF, ws=_ws())
    for kw in (dict(q=torch.zeros(B, D, H, dtype=BF).transpose(1, 2)), dict(lse=torch.zeros(H, B).T),
               dict(out=torch.zeros(H, B, D, dtype=BF).transpose(0, 1)), dict(block_table=i(3, B).T),
               dict(v_pages=torch.zeros(5, 64, G, D, dtype=BF).transpose(1, 2)), dict(seq_lens=i(2 * B)[::2])):
        a = _dense_args(**kw)
        a.pop("max_chunks")
        _refused(call, **a)


def _append_args(dtype=BF, **kw):
    z = lambda *s: torch.zeros(*s, dtype=dtype)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a = dict(k=z(9, G, D), v=z(9, G, D), k_pages=z(5, G, 64, D), v_pages=z(5, G, 64, D), block_table=i(B, 3),
             max_chunks=3, seq_lens=i(B), q=z(9, H, D), cu_new=i(B + 1), full_pages=i(B + 9 // 64))
    a.update(kw)
    return a


def test_append_arguments():
    sh = make_shape(B, H, G, D, 3 * 64, 0, HILS_BF16)
    z = lambda *s: torch.zeros(*s, dtype=BF)
    check_append_args(sh, **_append_args(q_out=z(9, H, D)))
    check_append_args(sh, **_append_args(k=z(B, G, D), v=z(B, G, D), q=z(B, H, D), cu_new=None))
    check_append_args(sh, **_append_args(k=z(B, G, 40, D), v=z(B, G, 40, D), q=z(B, H, 40, D), cu_new=None,
                                         new_lens=torch.zeros(B, dtype=torch.int32),
                                         full_pages=torch.zeros(B + 80 // 64, dtype=torch.int32)))
    check_append_args(make_shape(B, H, G, D, 3 * 64, 0, HILS_F32), **_append_args(torch.float32))
    call = hils.Append(B, H, G, D, 3, BF, inv_freq=torch.ones(16), ws=_ws())
    for a in (_append_args(), _append_args(q_out=z(9, H, D)), _append_args(q=None), _append_args(full_pages=None),
              _append_args(k=z(B, G, D), v=z(B, G, D), q=z(B, H, D), cu_new=None,
                           full_pages=torch.zeros(B, dtype=torch.int32)),
              _append_args(k=z(B, G, 40, D), v=z(B, G, 40, D), q=z(B, H, 40, D), cu_new=None,
                           full_pages=torch.zeros(B + 80 // 64, dtype=torch.int32))):
        a.pop("max_chunks")
        _right(call, **a)


@pytest.mark.parametrize("kw", [
    dict(k=torch.zeros(9, G, D)),
    dict(v=torch.zeros(8, G, D, dtype=BF)),
    dict(q=torch.zeros(9, G, D, dtype=BF)),
    dict(cu_new=None),                                     # nine rows for two sequences
    dict(cu_new=torch.zeros(B, dtype=torch.int32)),
    dict(cu_new=torch.zeros(B + 1, dtype=torch.int64)),
    dict(new_lens=torch.zeros(B, dtype=torch.int32)),      # packed rows have cu_new
    dict(k=torch.zeros(B, G, 9, D, dtype=BF), v=torch.zeros(B, G, 9, D, dtype=BF), q=None),  # cu_new with padded rows
    dict(k=torch.zeros(9, D, dtype=BF)),
    dict(k_pages=torch.zeros(5, G, 32, D, dtype=BF)),
    dict(v_pages=torch.zeros(4, G, 64, D, dtype=BF)),
    dict(block_table=torch.zeros(B, 4, dtype=torch.int32)),
    dict(block_table=torch.zeros(B, 3, dtype=torch.int64)),
    dict(seq_lens=torch.zeros(B + 1, dtype=torch.int32)),
    dict(full_pages=torch.zeros(B - 1, dtype=torch.int32)),
    dict(q=None, q_out=torch.zeros(9, H, D, dtype=BF)),
    dict(q_out=torch.zeros(9, H, D)),
])
def test_append_refuses(kw):
    with pytest.raises((ValueError, TypeError)):
        check_append_args(make_shape(B, H, G, D, 3 * 64, 0, HILS_BF16), **_append_args(**kw))
    a = _append_args(**kw)
    a.pop("max_chunks")
    _refused(hils.Append(B, H, G, D, 3, BF, ws=_ws()), **a)


def _dense_args(**kw):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)
    a = dict(q=torch.zeros(B, H, D, dtype=BF), k_pages=torch.zeros(5, G, 64, D, dtype=BF),
             v_pages=torch.zeros(5, G, 64, D, dtype=BF), block_table=i(B, 3), max_chunks=3, seq_lens=i(B))
    a.update(kw)
    return a


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(B, H, D)), dict(q=torch.zeros(B, G, D, dtype=BF)),
    dict(k_pages=torch.zeros(5, H, 64, D, dtype=BF)), dict(v_pages=torch.zeros(5, G, 64, D)),
    dict(k_pages=torch.zeros(5, G, D, dtype=BF)), dict(block_table=torch.zeros(B, 2, dtype=torch.int32)),
    dict(seq_lens=torch.zeros(B, dtype=torch.int64)), dict(out=torch.zeros(B, H, D)),
    dict(lse=torch.zeros(B, H, dtype=BF)), dict(lse=torch.zeros(B, H, 1)),
])
def test_dense_refuses(kw):
    sh = make_shape(B, H, G, D, 3 * 64, 0, HILS_BF16)
    check_dense_args(sh, **_dense_args())
    with pytest.raises((ValueError, TypeError)):
        check_dense_args(sh, **_dense_args(**kw))
    call = hils.DenseDecode(B, H, G, D, 3, BF, ws=_ws())
    a = _dense_args(**kw)
    a.pop("max_chunks")
    _refused(call, **a)
    a = _dense_args(out=torch.zeros(B, H, D, dtype=BF), lse=torch.zeros(B, H))
    a.pop("max_chunks")
    _right(call, **a)


def test_a_workspace_of_the_caller_is_checked():
    need = _abi.workspace_size(make_shape(B, H, G, D, 3 * 64, 0, HILS_BF16), hils.OP_DECODE_DENSE)
    hils.DenseDecode(B, H, G, D, 3, BF, ws=_ws(need))
    for ws in (_ws(need - 1), torch.zeros(need, dtype=torch.int32), _ws(2 * need)[::2]):
        with pytest.raises(ValueError):
            hils.DenseDecode(B, H, G, D, 3, BF, ws=ws)


def test_cache_calls_refuse_cpu_tensors_and_lengths_beyond_int32():
    with pytest.raises(ValueError):
        hils.rotate(torch.zeros(1, 1, 4, 64), torch.ones(32))
    with pytest.raises(ValueError):
        hils.decode_dense(torch.zeros(1, 1, 64), torch.zeros(1, 1, 64, 64), torch.zeros(1, 1, 64, 64),
                          torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        hils.DenseDecode(1, 1, 1, 64, 1 << 25, "bf16")
    with pytest.raises(ValueError):
        hils.Append(1, 1, 1, 64, 1 << 25, "bf16")


# ---- the C ABI's checks -----------------------------------------------------
def _sh(**kw):
    a = dict(batch=2, heads_q=8, heads_kv=2, head_dim=64, seq_len=640, top_k=0, dtype=1)
    a.update(kw)
    return make_shape(a["batch"], a["heads_q"], a["heads_kv"], a["head_dim"], a["seq_len"], a["top_k"], a["dtype"],
                      window=a.get("window", 0))


def test_rotate_rejects_before_launch():
    L, ref = hils.lib(), ctypes.byref
    s, r, ro = _sh(), Rows(1 << 20, 64, 64, 64), Rope(1 << 20, 32, 0)

    def call(s=s, q=r, k=r, rope=ro, ps=0, qo=r, ko=r, od=1):
        return L.hils_rotate(ref(s), q and ref(q), k and ref(k), rope and ref(rope), None, ps, 0, qo and ref(qo),
                             ko and ref(ko), od, None)

    assert call(q=None) == 1 and call(rope=None) == 1 and call(ko=None) == 1 and call(k=None) == 1
    assert call(od=7) == 1 and call(ps=-1) == 1
    assert call(q=Rows((1 << 20) + 8, 64, 64, 64)) == 1
    assert call(qo=Rows(1 << 20, 64, 64, 60)) == 1
    assert call(rope=Rope(None, 32, 0)) == 1 and call(rope=Rope(1 << 20, 80, 0)) == 1
    assert call(rope=Rope(1 << 20, 0, 0)) == 1 and call(rope=Rope(1 << 20, 32, 2)) == 1
    assert call(rope=Rope(1 << 20, 24, 0)) == 2
    assert call(s=_sh(head_dim=96)) == 2
    assert call(s=_sh(batch=0), q=None, qo=None) == 0 and call(s=_sh(seq_len=0)) == 0


def test_append_rejects_before_launch():
    L, ref = hils.lib(), ctypes.byref
    s, r, ro = _sh(), Rows(1 << 20, 64, 64, 64), Rope(1 << 20, 32, 0)

    def call(s=s, k=r, v=r, q=r, qo=r, n=4, cu=None, nl=None, sl=FAKE, bt=FAKE, mc=4, np_=4, rope=ro, kp=FAKE,
             vp=FAKE, fp=None, ws=FAKE, wsb=256):
        return L.hils_append_paged(ref(s), k and ref(k), v and ref(v), q and ref(q), qo and ref(qo), n, cu, nl, sl, bt,
                                   mc, np_, rope and ref(rope), kp, vp, fp, ws, wsb, None)

    assert call(k=None) == 1 and call(v=None) == 1 and call(q=None) == 1 and call(qo=None) == 1
    assert call(n=-1) == 1 and call(cu=FAKE, nl=FAKE) == 1 and call(sl=None) == 1 and call(bt=None) == 1
    assert call(mc=0) == 1 and call(np_=0) == 1 and call(kp=None) == 1 and call(vp=P_((1 << 20) + 4)) == 1
    assert call(k=Rows(1 << 20, 64, 4, 64)) == 1
    far = lambda i, h: Rows((i + 1) << 28, h * 4 * 64, 4 * 64, 64)
    good = dict(k=far(0, 2), v=far(1, 2), q=far(2, 8), qo=far(3, 8), kp=P_(5 << 28), vp=P_(6 << 28))
    assert call(**good, ws=None) == 3                                # nothing else is wrong with it
    assert call(**{**good, "vp": P_((5 << 28) + 16)}) == 1           # the pools overlap
    assert call(**{**good, "k": far(4, 2)}) == 1                     # keys read from the pool
    assert call(**{**good, "qo": far(0, 8)}) == 1                    # queries written over the keys
    assert call(**{**good, "qo": far(2, 8)}, ws=None) == 3           # in place
    assert call(**{**good, "qo": Rows(4 << 28, 4 * 64, 0, 64)}) == 1  # one row for every head
    assert call(rope=Rope(1 << 20, 24, 0)) == 2 and call(mc=1 << 26) == 2
    assert call(n=(1 << 31) - 1) == 2  # more rows than 32 bits count
    assert call(**good, wsb=128) == 3
    assert call(s=_sh(batch=0)) == 0 and call(n=0, k=None, v=None, q=None, qo=None, ws=None) == 0
    n = ctypes.c_size_t(0)
    assert L.hils_workspace_size(ref(s), hils.OP_APPEND, ref(n)) == 0 and n.value >= 256


def test_dense_rejects_before_launch():
    L, ref = hils.lib(), ctypes.byref
    s = _sh()
    n = ctypes.c_size_t(0)
    assert L.hils_workspace_size(ref(s), hils.OP_DECODE_DENSE, ref(n)) == 0 and n.value >= 256
    size = n.value

    def call(s=s, q=FAKE, k=FAKE, v=FAKE, bt=FAKE, mc=10, sl=FAKE, np_=4, out=FAKE, ws=FAKE, wsb=size):
        return L.hils_decode_dense(ref(s), q, k, v, bt, mc, sl, np_, out, None, ws, wsb, None)

    for name in ("q", "k", "v", "bt", "sl", "out"):
        assert call(**{name: None}) == 1, name
    assert call(mc=0) == 1 and call(mc=11) == 1 and call(np_=0) == 1
    assert call(q=P_((1 << 20) + 8)) == 1
    assert call(ws=None) == 3 and call(wsb=size - 1) == 3 and call(ws=P_((1 << 20) + 8)) == 3
    assert call(s=_sh(heads_q=6)) == 2 and call(s=_sh(window=100)) == 1
    assert call(s=_sh(batch=0)) == 0


# ---- rows that share memory -------------------------------------------------
def _rotate_status(q, k, qo, ko, h, g, n, b=2, d=64, dtype=1, out_dtype=1):
    """hils_rotate's status for rows at addresses that are never read: refused before the launch
    (1), or brought to a launch that finds no GPU (4)."""
    if torch.cuda.is_available():
        pytest.skip("an accepted call would be launched on the addresses")
    ref = lambda x: None if x is None else ctypes.byref(x)
    return hils.lib().hils_rotate(ref(_sh(batch=b, heads_q=h, heads_kv=g, head_dim=d, seq_len=n, dtype=dtype)), ref(q),
                                  ref(k), ref(Rope(1 << 20, 32, 0)), None, 0, 0, ref(qo), ref(ko), out_dtype, None)


def test_rotate_in_place_refuses_another_tensor_on_the_same_rows():
    """The header's promise: in place, the other tensor may lie between the rows, not on them."""
    n, base, far = 70, 1 << 20, 1 << 30
    dense = lambda p, h: Rows(p, h * n * 64, n * 64, 64)
    fused = lambda p, H: Rows(p, n * H * 64, 64, H * 64)  # a slice of [b, n, H, d]
    ok = lambda *a, **kw: _rotate_status(*a, n=n, **kw)
    q = dense(base, 2)
    assert ok(q, dense(base, 2), q, dense(far, 2), 2, 2) == 1               # k is q's memory
    assert ok(q, dense(base + 128, 2), q, dense(far, 2), 2, 2) == 1         # a row further on
    assert ok(q, q, q, q, 2, 2) == 1                                        # all four
    assert ok(dense(far, 2), dense(base, 2), dense(base, 2), dense(base, 2), 2, 2) == 1  # q_out on k in place
    assert ok(dense(base, 2), dense(far, 2), dense(far + (1 << 26), 2), dense(base + 64, 2), 2, 2) == 1
    # slices of one fused tensor, both in place
    f = lambda i: fused(base + i * 128, 12)
    assert ok(f(0), f(8), f(0), f(8), 8, 2) == 4                            # the model's own layout
    assert ok(f(0), f(7), f(0), f(7), 8, 2) == 1                            # a head too early
    assert ok(f(0), f(11), f(0), f(11), 8, 2) == 1                          # its second head is the next token's first
    assert ok(f(0), fused(base + 8 * 128, 11), f(0), fused(base + 8 * 128, 11), 8, 2) == 1  # of another width


def _append_status(q, qo, k, v, h, g, n, cu=FAKE):
    """hils_append_paged's status without a workspace, which is looked at last (3: nothing else
    is wrong)."""
    ref = ctypes.byref
    return hils.lib().hils_append_paged(ref(_sh(heads_q=h, heads_kv=g)), ref(k), ref(v), ref(q), ref(qo), n, cu, None, FAKE,
                                        FAKE, 4, 4, None, P_(5 << 28), P_(6 << 28), None, None, 256, None)


def test_append_in_place_refuses_keys_and_values_on_the_queries_rows():
    base, far = 1 << 20, 1 << 26
    f = lambda i, H=12: Rows(base + i * 128, 0, 64, H * 64)  # packed slices of [tokens, H, d]
    for cu in (FAKE, None):  # packed; one row per sequence and head
        r = f if cu else lambda i, H=12: Rows(base + i * 128, H * 64, 64, 0)
        n = 9 if cu else 1
        assert _append_status(r(0), r(0), r(8), r(10), 8, 2, n, cu) == 3
        assert _append_status(r(0), r(0), r(7), r(10), 8, 2, n, cu) == 1
        assert _append_status(r(0), r(0), r(8), r(0), 8, 2, n, cu) == 1
        assert _append_status(r(0), r(0), r(8), r(11), 8, 2, n, cu) == 1   # the next token's queries
        assert _append_status(r(0), r(0), Rows(far, 192, 64, 192), r(10), 8, 2, n, cu) == 3
    padded = lambda p, h, n: Rows(p, h * n * 64, n * 64, 64)
    assert _append_status(padded(base, 4, 9), padded(base, 4, 9), padded(base, 2, 9), padded(far, 2, 9), 4, 2, 9, None) == 1
    assert _append_status(padded(base, 4, 9), padded(base, 4, 9), padded(far, 2, 9), padded(2 * far, 2, 9), 4, 2, 9, None) == 3


def test_rotate_takes_outputs_that_lie_between_one_another():
    """dq and dk rotated back into the slices of one fused gradient, in the layouts that a model
    has it in."""
    n, base, out = 70, 1 << 20, 1 << 30
    dense = lambda p, h: Rows(p, h * n * 64, n * 64, 64)
    q, k = dense(base, 8), dense(base + (1 << 24), 2)
    tok = lambda i, H=12: Rows(out + i * 128, n * H * 64, 64, H * 64)          # [b, n, h + 2g, d]
    head = lambda i, H=12: Rows(out + i * n * 128, n * H * 64, n * 64, 64)     # [b, h + 2g, n, d]
    ok = lambda *a, **kw: _rotate_status(*a, n=n, **kw)
    assert ok(q, k, tok(0), tok(8), 8, 2) == 4 and ok(q, k, tok(4), tok(2), 8, 2) == 4
    assert ok(q, k, head(0), head(8), 8, 2) == 4
    assert ok(q, k, tok(0), tok(7), 8, 2) == 1 and ok(q, k, head(1), head(8), 8, 2) == 1
    assert ok(q, k, tok(0), tok(11), 8, 2) == 1 and ok(q, k, tok(0), head(0), 8, 2) == 1
    # [b, n, h, 3, d]: a head's q, k and v side by side; from it in place, and into it
    trio = lambda p, i: Rows(p + i * 128, n * 24 * 64, 192, 24 * 64)
    for o in (base, out):
        assert ok(trio(base, 0), trio(base, 1), trio(o, 0), trio(o, 1), 8, 8) == 4
        assert ok(trio(base, 0), trio(base, 1), trio(o, 0), trio(o, 0), 8, 8) == 1
    assert ok(trio(base, 0), trio(base, 1), trio(base, 2), trio(out, 1), 8, 8) == 4  # over the values
    assert ok(trio(base, 0), trio(base, 1), trio(base, 1), trio(out, 1), 8, 8) == 1
    # bf16 rows between fp32 ones: taken to share, and apart
    assert ok(tok(0), tok(8), Rows(out, 0, 64, 12 * 32), dense(base, 2), 8, 2, out_dtype=0) == 1
    assert ok(q, k, dense(out, 8), Rows(out + 8 * n * 64 * 4 * 2, 2 * n * 64, n * 64, 64), 8, 2, out_dtype=0) == 4


def test_rotate_accepts_no_rows_that_share_an_element():
    """Random rows against the elements they cover."""
    rng = np.random.RandomState(0)
    cover = lambda r, h, b, n: {r.data // 16 + (i * r.batch_stride + j * r.head_stride + t * r.token_stride) // 8 + e
                                for i in range(b) for j in range(h) for t in range(n) for e in range(8)}
    taken = {1: 0, 4: 0}
    for _ in range(1500):
        b, g, n = (int(x) for x in rng.randint(1, 4, 3))
        h = g * int(rng.choice([1, 2]))
        H = int(rng.randint(h + g, h + 3 * g + 1))
        perm = rng.permutation(3)
        size = [b, H, n]
        stride, s = [0, 0, 0], 64
        for i in perm:
            stride[i] = s
            s *= size[i]
        rows = lambda i, j=0: Rows((1 << 20) + i * stride[1] * 2 + j * 16, *stride)
        qo, ko = rows(int(rng.randint(0, H))), rows(int(rng.randint(0, H)), int(rng.choice([0, 0, 0, 1, 7])))
        if rng.rand() < 0.2:
            ko.token_stride += 64 * int(rng.randint(1, 9))
        far = lambda p, h: Rows(p, h * n * 64, n * 64, 64)
        st = _rotate_status(far(1 << 28, h), far(1 << 29, g), qo, ko, h, g, n, b=b)
        whole = [cover(qo, h, b, n), cover(ko, g, b, n)]
        if st == 4:
            assert not whole[0] & whole[1] and all(len(c) == 8 * x * b * n for c, x in zip(whole, (h, g)))
        else:
            assert st == 1
            if ko.token_stride == qo.token_stride or n == 1 or whole[0] & whole[1]:
                assert whole[0] & whole[1] or len(whole[0]) < 8 * h * b * n or len(whole[1]) < 8 * g * b * n
        taken[st] += 1
    assert min(taken.values()) > 200


def test_kernels_that_start_early_read_through_the_ordinary_path():
    """A kernel that may run beside its predecessor (wait_for_stream) must not use loads that ask
    for data nobody writes during its life."""
    import pathlib
    src = pathlib.Path(_abi.__file__).parent / "csrc"
    early = [p for p in sorted(src.glob("*.cu")) if "wait_for_stream();" in p.read_text()]
    assert {p.name for p in early} >= {"decode_dense.cu", "rotate.cu"}
    for p in early:
        for word in ("__ldg(", "ld.global.nc", "__restrict__"):
            assert word not in p.read_text(), f"{p.name}: {word}"


def test_dense_takes_any_window():
    """The limit of 128 chunks is the prefill kernels'."""
    L, ref, n = hils.lib(), ctypes.byref, ctypes.c_size_t(0)
    for w, other in ((64 * 128, 0), (64 * 129, 2), (1 << 30, 2)):
        s = _sh(window=w, seq_len=640)
        assert L.hils_workspace_size(ref(s), hils.OP_DECODE_DENSE, ref(n)) == 0
        assert L.hils_decode_dense(ref(s), FAKE, FAKE, FAKE, FAKE, 10, FAKE, 4, FAKE, None, None, n.value, None) == 3
        for op in (hils.OP_ATTEND, hils.OP_DECODE, hils.OP_APPEND):
            assert L.hils_workspace_size(ref(s), op, ref(n)) == other


def test_int_arrays_off_their_alignment_are_refused():
    """A 4-byte load from such an address would fault on the GPU."""
    L, ref, odd = hils.lib(), ctypes.byref, P_((1 << 20) + 2)
    s, ro = _sh(), Rope(1 << 20, 32, 0)
    far = lambda i, h: Rows((i + 1) << 28, h * 4 * 64, 4 * 64, 64)
    k, v = far(0, 2), far(1, 2)

    def append(cu=None, nl=None, sl=FAKE, bt=FAKE, fp=None):
        return L.hils_append_paged(ref(s), ref(k), ref(v), None, None, 4, cu, nl, sl, bt, 4, 4, ref(ro), P_(5 << 28),
                                   P_(6 << 28), fp, None, 256, None)

    assert append() == 3 and append(nl=FAKE, fp=FAKE) == 3 and append(cu=FAKE) == 3
    assert [append(**{x: odd}) for x in ("cu", "nl", "sl", "bt", "fp")] == [1] * 5
    n = ctypes.c_size_t(0)
    L.hils_workspace_size(ref(s), hils.OP_DECODE_DENSE, ref(n))

    def dense(bt=FAKE, sl=FAKE, lse=None):
        return L.hils_decode_dense(ref(s), P_(1 << 28), P_(2 << 28), P_(3 << 28), bt, 10, sl, 4, P_(4 << 28), lse, None,
                                   n.value, None)

    assert dense() == 3 and dense(lse=P_(5 << 28)) == 3
    assert [dense(**{x: odd}) for x in ("bt", "sl", "lse")] == [1] * 3
    r = Rows(1 << 28, 8 * 640 * 64, 640 * 64, 64)
    assert L.hils_rotate(ref(s), ref(r), None, ref(ro), odd, 0, 0, ref(r), None, 1, None) == 1


def test_rotate_refuses_one_tensor_without_heads():
    q, k, f = torch.zeros(B, H, N, D, dtype=BF), torch.zeros(B, G, N, D, dtype=BF), torch.ones(16)
    _refused(hils.rotate, q, f, k=k[:, :0])
    _refused(hils.rotate, q[:, :0], f, k=k)
    assert hils.rotate(q[:, :0], f).shape == (B, 0, N, D)
    assert [x.shape[1] for x in hils.rotate(q[:, :0], f, k=k[:, :0])] == [0, 0]


def test_dense_refuses_outputs_on_its_inputs():
    L, ref, n = hils.lib(), ctypes.byref, ctypes.c_size_t(0)
    s = _sh()  # q and out 2 KB, a pool of four pages 64 KB, lse 64 bytes
    L.hils_workspace_size(ref(s), hils.OP_DECODE_DENSE, ref(n))

    def call(out=5 << 20, lse=None, q=1 << 20):
        return L.hils_decode_dense(ref(s), P_(q), P_(2 << 20), P_(3 << 20), FAKE, 10, FAKE, 4, P_(out),
                                   lse and P_(lse), None, n.value, None)

    assert call() == 3 and call(out=1 << 20) == 3 and call(lse=6 << 20) == 3
    assert call(out=(5 << 20) - 16, lse=(5 << 20) + 2032) == 3
    for kw in (dict(out=(1 << 20) + 16), dict(out=(1 << 20) - 16), dict(out=2 << 20), dict(out=(3 << 20) + 65520),
               dict(lse=5 << 20), dict(lse=(5 << 20) + 2044), dict(lse=(1 << 20) + 4), dict(lse=2 << 20),
               dict(out=1 << 20, lse=(1 << 20) + 64)):
        assert call(**kw) == 1, kw
