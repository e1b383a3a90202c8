"""Packed-batch calls: QK norm, dense attention, linear attention (prompts and
single tokens) and decode over a shared prefix, against plain float64 forms.

Tolerances, element by element, from the roundings the kernels make (half a
step: bf16 2^-8, relative):
  * a bf16 output is rounded once: 2^-8 |ref|;
  * attention rounds each softmax weight to bf16 before the product with V, so
    its sum is off by at most 2^-8 sum p |v|; the weights themselves carry the
    exponential's 1e-4 and the logits' fp32 error, together below 2^-11 (logits
    of rows of root mean square 1 stay below sqrt(d) = 11.4, an error of
    d 2^-24 relative to sum |q k| changes a weight by less than 1e-4);
  * linear attention rounds the state (2^-8 |S|) and the masked products
    (2^-8 |q k|) to bf16: at most 2^-8 |q| Sabs with Sabs the recurrence of the
    absolute values.  Norm-wise these three independent roundings (each at most
    2^-8, root mean square below 2^-9 2/sqrt(3)) stay below 2^-8;
  * states take decayed values split into three bf16 parts (2^-24), and fp32 sums
    of up to 3 x 128 terms per tile on the tensor core, which may round towards
    zero (2^-23 each): 2^-23 x 384 Sabs is below 2^-14, in practice far below:
    terms of both signs cancel in their roundings.  Element-wise 2^-16 Sabs is
    asked for, norm-wise 2^-20.
"""
import ctypes
import json
import math
import os
import subprocess
import sys

import pytest
import torch

sala = pytest.importorskip("hybrid_sparse_linear_lightning_b200.sala")

FAKE = ctypes.c_void_p(0x10000)
MISALIGNED = ctypes.c_void_p(0x10008)
BF = torch.bfloat16
HALF = 2.0 ** -8


# ------------------------------------------------------------------------------------ references

def ref_qk_norm(x, w, pos, eps=1e-6, base=10000.0):
    x = x.double()
    d = x.shape[-1]
    y = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    if pos is None:
        return y, torch.zeros_like(y)
    i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
    a = pos.double()[:, None, None] * base ** (-2.0 * i / d)
    lo, hi = y[..., : d // 2], y[..., d // 2:]
    mag = lo.abs() + hi.abs()
    return (torch.cat([lo * a.cos() - hi * a.sin(), hi * a.cos() + lo * a.sin()], -1),
            torch.cat([mag, mag], -1))


def softmax_v(q, k, v, n_seen, scale):
    """q [R, d], k and v [n, d], row r seeing n_seen[r] keys: (softmax v, softmax |v|)."""
    x = q @ k.T * scale
    x = x.masked_fill(torch.arange(k.shape[0], device=q.device)[None] >= n_seen[:, None], -math.inf)
    p = torch.softmax(x, -1)
    keep = torch.where(p > 0, p, 0.0)
    return keep @ v, keep @ v.abs()


def ref_dense(q, k, v, gate, cu, scale=None):
    T, Hq, d = q.shape
    G = Hq // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    o = torch.full((T, Hq, d), math.nan, dtype=torch.float64, device=q.device)
    a = o.clone()
    for s, e in zip(cu[:-1], cu[1:]):
        if e <= s:
            continue
        seen = torch.arange(1, e - s + 1, device=q.device)
        for h in range(Hq):
            o[s:e, h], a[s:e, h] = softmax_v(q[s:e, h].double(), k[s:e, h // G].double(),
                                             v[s:e, h // G].double(), seen, scale)
    sg = torch.sigmoid(gate.double())
    return o * sg, a * sg


def ref_linear(q, k, v, gate, lam, cu, states, scale=1.0):
    """states: list of [H, d, d] (or None).  (out, bound, final states, their absolute recurrences)"""
    T, H, d = q.shape
    out = torch.full((T, H, d), math.nan, dtype=torch.float64, device=q.device)
    mag = out.clone()
    fin, fabs = [], []
    L = lam.double()[:, None, None]
    for i, (s, e) in enumerate(zip(cu[:-1], cu[1:])):
        S = torch.zeros((H, d, d), dtype=torch.float64, device=q.device) if states[i] is None else states[i].double()
        A = S.abs()
        for t in range(s, e):
            kk, vv, qq = k[t].double(), v[t].double(), q[t].double()
            S = L * S + kk[:, :, None] * vv[:, None, :]
            A = L * A + kk.abs()[:, :, None] * vv.abs()[:, None, :]
            out[t] = (qq[:, None, :] @ S)[:, 0] * scale
            mag[t] = (qq.abs()[:, None, :] @ A)[:, 0] * abs(scale)
        fin.append(S)
        fabs.append(A)
    sg = torch.sigmoid(gate.double())
    return out * sg, mag * sg, fin, fabs


def ref_prefix(q, k, v, gate, pk, pv, kc, vc, lens, slots, scale=None):
    B, Hq, d = q.shape
    Hkv = k.shape[1]
    G = Hq // Hkv
    scale = d ** -0.5 if scale is None else scale
    o = torch.full((B, Hq, d), math.nan, dtype=torch.float64, device=q.device)
    a = o.clone()
    for b in range(B):
        if slots[b] < 0:
            continue
        n = lens[b]
        for g in range(Hkv):
            parts_k = [kc[slots[b], :n, g].double(), k[b, g:g + 1].double()]
            parts_v = [vc[slots[b], :n, g].double(), v[b, g:g + 1].double()]
            if pk is not None:
                parts_k.insert(0, pk[:, g].double())
                parts_v.insert(0, pv[:, g].double())
            kk, vv = torch.cat(parts_k), torch.cat(parts_v)
            rows = slice(g * G, (g + 1) * G)
            o[b, rows], a[b, rows] = softmax_v(q[b, rows].double(), kk, vv,
                                               torch.full((G,), kk.shape[0], device=q.device), scale)
    sg = torch.sigmoid(gate.double())
    return o * sg, a * sg


def check(got, ref, tol, what=""):
    err = (got.double() - ref).abs()
    bad = ~(err <= tol)
    assert not bool(bad.any()), (what, int(bad.sum()), float((err / tol.clamp_min(1e-300)).nan_to_num(1e30).max()))


def attn_tol(ref, mag):
    return HALF * ref.abs() + (HALF * (1 + HALF) + 2.0 ** -11) * mag + 1e-30


def clean(stream=None):
    torch.cuda.synchronize()
    assert sala.sala_get_device_status(stream) == sala.SALA_OK


# ----------------------------------------------------------------------------------------- inputs

def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF)


def unit(g, *shape):
    x = torch.randn(shape, generator=g, device="cuda")
    return (x * torch.rsqrt(x.square().mean(-1, keepdim=True))).to(BF)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def starts(lens, first=0):
    cu = [first]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def decays(H):
    return torch.tensor([1.0 - 2.0 ** (-5.0 - h / 4.0) for h in range(H)], device="cuda")


def dense_inputs(T, Hq, Hkv, d, seed=0):
    g = gen(seed)
    return unit(g, T, Hq, d), unit(g, T, Hkv, d), rnd(g, T, Hkv, d), rnd(g, T, Hq, d)


def linear_inputs(T, H, d, seed=0):
    g = gen(seed)
    return unit(g, T, H, d), unit(g, T, H, d), rnd(g, T, H, d), rnd(g, T, H, d)


# -------------------------------------------------------------------------------- refusals (CPU)

def raw(fn, d, *args):
    return getattr(sala.LIB, fn)(ctypes.byref(d) if d is not None else None, *args, None)


def qk_desc(**kw):
    b = dict(tokens=8, q_heads=4, k_heads=1, head_dim=64, dtype=sala.SALA_BF16, rope_base=1e4, rms_eps=1e-6)
    b.update(kw)
    return sala.QkNormDesc(*b.values())


def dense_desc(**kw):
    b = dict(tokens=8, n_seqs=1, q_heads=4, kv_heads=1, head_dim=64, dtype=sala.SALA_BF16, scale=0.0)
    b.update(kw)
    return sala.DenseDesc(*b.values())


def lin_desc(**kw):
    b = dict(tokens=8, n_seqs=8, n_slots=8, heads=4, head_dim=64, dtype=sala.SALA_BF16, scale=1.0)
    b.update(kw)
    return sala.PackedLinearDesc(*b.values())


def prefix_desc(**kw):
    b = dict(batch=2, prefix_len=10, n_slots=2, q_heads=4, kv_heads=1, head_dim=64, cache_capacity=64,
             dtype=sala.SALA_BF16, scale=0.0)
    b.update(kw)
    return sala.PrefixDesc(*b.values())


BIG = 1 << 40


@pytest.mark.parametrize("kw,ptr,want", [
    (dict(tokens=0), FAKE, "INVALID_ARG"), (dict(k_heads=0), FAKE, "INVALID_ARG"),
    (dict(dtype=7), FAKE, "INVALID_ARG"), (dict(rms_eps=-1.0), FAKE, "INVALID_ARG"),
    (dict(rope_base=0.0), FAKE, "INVALID_ARG"), (dict(head_dim=96), FAKE, "UNSUPPORTED"),
    (dict(q_heads=9000), FAKE, "UNSUPPORTED"), (dict(), None, "INVALID_ARG"),
    (dict(), MISALIGNED, "INVALID_ARG")])
def test_qk_norm_refusals(kw, ptr, want):
    assert raw("sala_qk_norm", qk_desc(**kw), ptr, ptr, ptr, ptr, None, ptr, ptr) == \
        getattr(sala, "SALA_ERR_" + want)


@pytest.mark.parametrize("kw,ptr,want", [
    (dict(tokens=0), FAKE, "INVALID_ARG"), (dict(n_seqs=0), FAKE, "INVALID_ARG"),
    (dict(q_heads=6, kv_heads=4), FAKE, "INVALID_ARG"), (dict(scale=math.nan), FAKE, "INVALID_ARG"),
    (dict(head_dim=80), FAKE, "UNSUPPORTED"), (dict(q_heads=129), FAKE, "UNSUPPORTED"),
    (dict(dtype=sala.SALA_F32), FAKE, "UNSUPPORTED"), (dict(), None, "INVALID_ARG"),
    (dict(), MISALIGNED, "INVALID_ARG")])
def test_dense_refusals(kw, ptr, want):
    assert raw("sala_dense_prefill", dense_desc(**kw), ptr, ptr, ptr, ptr, ptr, ptr, FAKE, BIG) == \
        getattr(sala, "SALA_ERR_" + want)
    if kw:
        assert sala.LIB.sala_dense_workspace_size(ctypes.byref(dense_desc(**kw))) == 0


@pytest.mark.parametrize("kw,ptr,want", [
    (dict(tokens=0), FAKE, "INVALID_ARG"), (dict(heads=0), FAKE, "INVALID_ARG"),
    (dict(n_slots=0), FAKE, "INVALID_ARG"), (dict(n_slots=7), FAKE, "INVALID_ARG"),
    (dict(scale=math.inf), FAKE, "INVALID_ARG"), (dict(head_dim=32), FAKE, "UNSUPPORTED"),
    (dict(), None, "INVALID_ARG"), (dict(), MISALIGNED, "INVALID_ARG")])
def test_packed_linear_refusals(kw, ptr, want):
    want = getattr(sala, "SALA_ERR_" + want)
    d = lin_desc(**kw)
    assert raw("sala_linear_packed_prefill", d, ptr, ptr, ptr, ptr, ptr, ptr, None, None, None, ptr, FAKE,
               BIG) == want
    assert raw("sala_linear_packed_step", d, ptr, ptr, ptr, ptr, ptr, None, ptr, ptr) == want


def test_packed_linear_refusals_of_one_form():
    assert raw("sala_linear_packed_prefill", lin_desc(dtype=sala.SALA_F32), *[FAKE] * 6, None, None, None, FAKE,
               FAKE, BIG) == sala.SALA_ERR_UNSUPPORTED
    assert raw("sala_linear_packed_step", lin_desc(tokens=9), *[FAKE] * 5, None, FAKE, FAKE) == \
        sala.SALA_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,ptr,want", [
    (dict(batch=0), FAKE, "INVALID_ARG"), (dict(prefix_len=-1), FAKE, "INVALID_ARG"),
    (dict(n_slots=1), FAKE, "INVALID_ARG"), (dict(cache_capacity=0), FAKE, "INVALID_ARG"),
    (dict(q_heads=6, kv_heads=4), FAKE, "INVALID_ARG"), (dict(head_dim=256), FAKE, "UNSUPPORTED"),
    (dict(q_heads=258, kv_heads=2), FAKE, "UNSUPPORTED"), (dict(dtype=sala.SALA_F32), FAKE, "UNSUPPORTED"),
    (dict(cache_capacity=1 << 31), FAKE, "UNSUPPORTED"), (dict(), None, "INVALID_ARG"),
    (dict(), MISALIGNED, "INVALID_ARG")])
def test_prefix_refusals(kw, ptr, want):
    assert raw("sala_prefix_decode", prefix_desc(**kw), *[ptr] * 9, None, ptr, FAKE, BIG) == \
        getattr(sala, "SALA_ERR_" + want)


def test_null_descriptors():
    assert raw("sala_qk_norm", None, *[FAKE] * 7) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_dense_prefill", None, *[FAKE] * 7, BIG) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_linear_packed_prefill", None, *[FAKE] * 11, BIG) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_linear_packed_step", None, *[FAKE] * 8) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_prefix_decode", None, *[FAKE] * 12, BIG) == sala.SALA_ERR_INVALID_ARG


def test_workspaces_too_small_are_refused():
    for fn, size, d, n in (("sala_dense_prefill", "sala_dense_workspace_size", dense_desc(tokens=500, n_seqs=3), 6),
                           ("sala_linear_packed_prefill", "sala_linear_packed_workspace_size",
                            lin_desc(tokens=9000, n_seqs=3, heads=32, head_dim=128), 10),
                           ("sala_prefix_decode", "sala_prefix_workspace_size", prefix_desc(), 11)):
        need = getattr(sala.LIB, size)(ctypes.byref(d))
        if need:
            assert raw(fn, d, *[FAKE] * n, FAKE, need - 1) == sala.SALA_ERR_WORKSPACE
            assert raw(fn, d, *[FAKE] * n, None, need) == sala.SALA_ERR_WORKSPACE
            assert raw(fn, d, *[FAKE] * n, MISALIGNED, need) in (sala.SALA_ERR_INVALID_ARG, sala.SALA_ERR_WORKSPACE)


def test_helpers_refuse_wrong_tensors():
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="k_norm"):
        sala.dense_prefill(z(4, 2, 64), z(4, 1, 32), z(4, 1, 64), z(4, 2, 64), cu)
    with pytest.raises(ValueError, match="v"):
        sala.dense_prefill(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64, dt=torch.float32), z(4, 2, 64), cu)
    with pytest.raises(ValueError, match="cu_seqlens"):
        sala.dense_prefill(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), z(4, 2, 64), cu.long())
    with pytest.raises(ValueError, match="contiguous"):
        sala.dense_prefill(z(2, 4, 64).transpose(0, 1), z(4, 1, 64), z(4, 1, 64), z(4, 2, 64), cu)
    with pytest.raises(ValueError, match="CUDA device"):
        sala.dense_prefill(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), z(4, 2, 64), cu)
    with pytest.raises(ValueError, match="positions"):
        sala.qk_norm(z(4, 2, 64), z(4, 1, 64), z(64, dt=torch.float32), z(64, dt=torch.float32),
                     torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="state"):
        sala.linear_packed_step(z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(4, 2, 64), z(2, dt=torch.float32),
                                z(4, 2, 64, 64))
    with pytest.raises(ValueError, match="both"):
        sala.prefix_decode(z(1, 2, 64), z(1, 1, 64), z(1, 1, 64), z(1, 2, 64), z(4, 1, 64), None, z(1, 8, 1, 64),
                           z(1, 8, 1, 64), torch.zeros(1, dtype=torch.int32))


# ---------------------------------------------------------------------------------------- QK norm

@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hk,d", [(1, 1, 1, 64), (7, 4, 1, 128), (2050, 7, 3, 64), (2049, 32, 2, 128)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("rope", [False, True])
def test_qk_norm(cuda_device, T, Hq, Hk, d, dtype, rope):
    g = gen(T)
    q = (3 * torch.randn((T, Hq, d), generator=g, device="cuda")).to(dtype)
    k = torch.randn((T, Hk, d), generator=g, device="cuda").to(dtype)
    wq, wk = (1 + 0.1 * torch.randn((d,), generator=g, device="cuda") for _ in range(2))
    pos = torch.randint(-5, (1 << 31) - 1, (T,), generator=g, device="cuda", dtype=torch.int64).int() if rope else None
    q0 = q.clone()
    qn, kn = sala.qk_norm(q, k, wq, wk, pos)
    clean()
    assert torch.equal(q, q0) and qn.dtype == kn.dtype == BF
    for got, x, w in ((qn, q, wq), (kn, k, wk)):
        ref, mag = ref_qk_norm(x, w, pos)
        # angles up to 2^31 are formed in fp64 from frequencies an ulp off, here and there: 2^31 4 2^-53 = 2^-20;
        # reduced they are rounded to fp32 (2^-24 pi), sine and cosine are 2 ulp off, the norm 4 ulp
        check(got, ref, HALF * ref.abs() + 2.0 ** -19 * (mag + ref.abs()) + 1e-30)


@pytest.mark.gpu
def test_qk_norm_in_place_zero_rows_and_bad_rows(cuda_device):
    g = gen(3)
    q, k = rnd(g, 5, 4, 128), rnd(g, 5, 2, 128)
    w = torch.ones(128, device="cuda")
    want = sala.qk_norm(q, k, w, w, i32([0, 1, 2, 3, 4]))
    q[2] = 0
    k[1, 0, 7] = math.nan
    q[3, 1, 5] = math.inf
    got = sala.qk_norm(q, k, w, w, i32([0, 1, 2, 3, 4]), outs=(q, k))
    clean()
    assert got[0] is q and bool((q[2] == 0).all())
    assert bool(k[1, 0].isnan().all()) and torch.equal(k[1, 1], want[1][1, 1]) and torch.equal(k[0], want[1][0])
    assert not bool(q[3, 1].isfinite().all()) and torch.equal(q[3, 2:], want[0][3, 2:]) and torch.equal(q[4], want[0][4])


# ----------------------------------------------------------------------------------------- dense

DENSE = [([1], 1, 1, 64), ([5], 4, 1, 64), ([0, 3, 0, 1, 130], 4, 2, 128), ([127, 128, 129], 6, 2, 64),
         ([257, 1, 64, 300], 16, 1, 128), ([513], 7, 1, 128), ([70, 700], 3, 3, 128), ([40, 9], 128, 1, 64),
         ([90], 100, 1, 128), ([1025, 255], 8, 8, 64)]


@pytest.mark.gpu
@pytest.mark.parametrize("lens,Hq,Hkv,d", DENSE)
def test_dense_prefill(cuda_device, lens, Hq, Hkv, d):
    before, behind = 3, 5                        # rows that belong to no sequence
    cu = starts(lens, before)
    T = cu[-1] + behind
    q, k, v, gate = dense_inputs(T, Hq, Hkv, d, seed=sum(lens))
    out = torch.full((T, Hq, d), 7.0, dtype=BF, device="cuda")
    assert sala.dense_prefill(q, k, v, gate, i32(cu), out=out) is out
    clean()
    ref, mag = ref_dense(q, k, v, gate, cu)
    check(out[before:cu[-1]], ref[before:cu[-1]], attn_tol(ref, mag)[before:cu[-1]])
    assert bool((out[:before] == 7).all()) and bool((out[cu[-1]:] == 7).all())


@pytest.mark.gpu
def test_dense_scale_and_large_logits(cuda_device):
    """Logits far apart: the running maximum grows block after block, so old sums are rescaled."""
    T, d = 900, 64
    q, k, v, gate = dense_inputs(T, 2, 1, d, seed=5)
    k = (k.float() * torch.linspace(0.1, 6.0, T, device="cuda")[:, None, None]).to(BF)
    out = sala.dense_prefill(q, k, v, gate, i32([0, T]), scale=0.5)
    clean()
    ref, mag = ref_dense(q, k, v, gate, [0, T], scale=0.5)
    # logits reach 6 * 64 * 0.5 = 192: their fp32 error d 2^-24 * 192 stays below 2^-10
    check(out, ref, attn_tol(ref, mag) + 2.0 ** -9 * mag)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_dense_isolation(cuda_device, bad):
    """NaN or infinity in one sequence's tokens reach no other sequence and no earlier token."""
    lens = [200, 130, 300]
    cu = starts(lens)
    q, k, v, gate = dense_inputs(cu[-1], 8, 2, 128, seed=9)
    want = sala.dense_prefill(q, k, v, gate, i32(cu))
    u = cu[1] + 70
    for t in (k, v):
        t[u, 0, 5] = bad
    q[u, 1] = bad
    k[cu[2], 1], v[cu[2], 1] = bad, bad
    got = sala.dense_prefill(q, k, v, gate, i32(cu))
    clean()
    G = 4
    ok = torch.ones_like(want, dtype=torch.bool)
    ok[u:cu[2], :G] = False          # from token u on, kv head 0
    ok[cu[2]:, G:] = False           # the whole third sequence, kv head 1
    ok[u, 1] = False
    assert torch.equal(got[ok], want[ok])
    assert not bool(got[u:cu[2], 0, 5].isfinite().any())
    assert not bool(got[cu[2]:, G:].isfinite().any())


@pytest.mark.gpu
def test_dense_value_only_nonfinite(cuda_device):
    q, k, v, gate = dense_inputs(300, 4, 1, 64, seed=2)
    want = sala.dense_prefill(q, k, v, gate, i32([0, 300]))
    v[290, 0, 3] = math.inf
    got = sala.dense_prefill(q, k, v, gate, i32([0, 300]))
    clean()
    assert torch.equal(got[:290], want[:290])
    assert bool((got[290:, :, 3] == math.inf).all())
    keep = [c for c in range(64) if c != 3]
    assert torch.equal(got[290:, :, keep], want[290:, :, keep])


@pytest.mark.gpu
@pytest.mark.parametrize("cu", [[0, 5, 3, 10], [0, 4, 99], [-2, 4, 10]])
def test_dense_bad_bounds_set_the_status(cuda_device, cu):
    T = 10
    q, k, v, gate = dense_inputs(T, 2, 1, 64)
    out = torch.full((T, 2, 64), 7.0, dtype=BF, device="cuda")
    sala.dense_prefill(q, k, v, gate, i32(cu), out=out)
    torch.cuda.synchronize()
    assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
    assert sala.sala_get_device_status() == sala.SALA_OK
    good = [(a, b) for a, b in zip(cu[:-1], cu[1:]) if 0 <= a <= b <= T]
    if cu == [0, 4, 99] or cu == [-2, 4, 10]:
        a, b = good[0]
        ref, mag = ref_dense(q, k, v, gate, [a, b])
        check(out[a:b], ref[a:b], attn_tol(ref, mag)[a:b])
        rest = torch.ones(T, dtype=torch.bool)
        rest[a:b] = False
        assert bool((out[rest] == 7).all())


@pytest.mark.gpu
def test_dense_is_deterministic_on_streams_and_in_graphs(cuda_device):
    lens = [300, 17, 200]
    cu = i32(starts(lens))
    q, k, v, gate = dense_inputs(sum(lens), 8, 2, 128, seed=1)
    want = sala.dense_prefill(q, k, v, gate, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    on_s = sala.dense_prefill(q, k, v, gate, cu, stream=s)
    s.synchronize()
    assert torch.equal(on_s, want)
    outs = [torch.zeros_like(want) for _ in range(2)]
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            sala.dense_prefill(q, k, v, gate, cu, out=o)
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)
    cu.copy_(i32([0, 100, 100, sum(lens)]))           # a replay follows what the lengths hold then
    again = sala.dense_prefill(q, k, v, gate, cu)
    graphs[0].replay()
    clean()
    assert torch.equal(outs[0], again) and not torch.equal(again, want)


# ---------------------------------------------------------------------------------------- linear

LINEAR = [([1], 1, 64), ([3, 0, 1], 4, 64), ([128], 2, 128), ([127, 129, 64], 3, 128), ([1000, 5], 2, 128),
          ([70, 333], 8, 64), ([2600], 1, 128), ([2100, 40, 1500], 3, 64)]


def lin_check(out, ref, mag):
    check(out, ref, HALF * ref.abs() + HALF * (1 + HALF) * mag + 1e-30)
    assert float((out.double() - ref).norm() / ref.norm()) < HALF


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,d", LINEAR)
@pytest.mark.parametrize("with_state", [False, True])
def test_linear_packed_prefill(cuda_device, lens, H, d, with_state):
    before, behind = 2, 3
    cu = starts(lens, before)
    T, n = cu[-1] + behind, len(lens)
    q, k, v, gate = linear_inputs(T, H, d, seed=sum(lens) + d)
    lam = decays(H)
    out = torch.full((T, H, d), 7.0, dtype=BF, device="cuda")
    pool, slots, fin_pool = None, None, None
    init = [None] * n
    if with_state:
        pool = torch.randn((n + 2, H, d, d), generator=gen(4), device="cuda")
        perm = torch.randperm(n + 2, generator=gen(6), device="cuda")[:n]
        slots = perm.int()
        init = [pool[p] for p in perm.tolist()]
        fin_pool = torch.full_like(pool, 3.0)
    ref, mag, fin, fabs = ref_linear(q, k, v, gate, lam, cu, init, scale=0.5)
    sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), slots=slots, state_in=pool, state_out=fin_pool,
                               scale=0.5, out=out)
    clean()
    lin_check(out[before:cu[-1]], ref[before:cu[-1]], mag[before:cu[-1]])
    assert bool((out[:before] == 7).all()) and bool((out[cu[-1]:] == 7).all())
    if with_state:
        for p, S, A in zip(slots.tolist(), fin, fabs):
            check(fin_pool[p], S, 2.0 ** -16 * A + 1e-30)
            assert float((fin_pool[p].double() - S).norm() / S.norm()) < 2.0 ** -20
        others = [i for i in range(n + 2) if i not in slots.tolist()]
        assert bool((fin_pool[others] == 3).all())
        sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), slots=slots, state_in=pool, state_out=pool,
                                   scale=0.5, out=torch.empty_like(out))        # in place
        clean()
        assert all(torch.equal(pool[p], fin_pool[p]) for p in slots.tolist())


@pytest.mark.gpu
@pytest.mark.parametrize("value", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("d", [64, 128])
def test_linear_packed_special_decays(cuda_device, value, d):
    cu = [0, 300, 420]
    q, k, v, gate = linear_inputs(420, 2, d, seed=1)
    lam = torch.full((2,), value, device="cuda")
    pool = torch.randn((2, 2, d, d), generator=gen(4), device="cuda")
    fin = torch.empty_like(pool)
    out = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool, state_out=fin)
    clean()
    ref, mag, S, A = ref_linear(q, k, v, gate, lam, cu, [pool[0], pool[1]])
    lin_check(out, ref, mag)
    for i in range(2):
        check(fin[i], S[i], 2.0 ** -16 * A[i] + 1e-30)


@pytest.mark.gpu
def test_linear_packed_slots(cuda_device):
    """Padded, doubled and out-of-range slots: the sequence starts from zeros and no entry is written."""
    cu = [0, 40, 80, 120, 160]
    q, k, v, gate = linear_inputs(160, 2, 64, seed=1)
    lam = decays(2)
    pool = torch.randn((2, 2, 64, 64), generator=gen(4), device="cuda")
    for slots, fault in (([1, -1, 0, -7], False), ([1, 1, 0, -1], True), ([1, 5, 0, -1], True)):
        fin = torch.full_like(pool, 3.0)
        out = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), slots=i32(slots), state_in=pool, state_out=fin)
        torch.cuda.synchronize()
        assert sala.sala_get_device_status() == (sala.SALA_ERR_DEVICE_FAULT if fault else sala.SALA_OK)
        ref, mag, S, A = ref_linear(q, k, v, gate, lam, cu, [pool[1], None, pool[0], None])
        lin_check(out, ref, mag)
        for i, p in ((0, 1), (2, 0)):
            check(fin[p], S[i], 2.0 ** -16 * A[i] + 1e-30)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_linear_packed_isolation(cuda_device, bad):
    cu = starts([200, 130, 300])
    q, k, v, gate = linear_inputs(cu[-1], 2, 128, seed=9)
    lam = decays(2)
    pool = torch.randn((3, 2, 128, 128), generator=gen(4), device="cuda")
    a, b = torch.empty_like(pool), torch.empty_like(pool)
    want = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool, state_out=a)
    u = cu[1] + 50
    v[u, 0, 5] = bad
    k[u + 3, 1, 2] = bad
    v[cu[2], 1] = bad
    got = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool, state_out=b)
    clean()
    ok = torch.ones_like(want, dtype=torch.bool)
    ok[u:cu[2], 0, 5] = False
    ok[u + 3:cu[2], 1] = False
    ok[cu[2]:, 1] = False
    assert torch.equal(got[ok], want[ok])
    assert not bool(got[u:cu[2], 0, 5].isfinite().any())
    assert not bool(got[u + 3:cu[2], 1].isfinite().any()) and not bool(got[cu[2]:, 1].isfinite().any())
    assert torch.equal(a[0], b[0]) and torch.equal(a[2, 0], b[2, 0])
    assert not bool(b[1, 0, :, 5].isfinite().any()) and torch.equal(a[1, 0, :, :5], b[1, 0, :, :5])


@pytest.mark.gpu
def test_linear_packed_heads_side_by_side(cuda_device):
    """Two heads of 64 share a tile: NaN in one leaves the other's bits as they are."""
    cu = [0, 150, 200]
    q, k, v, gate = linear_inputs(200, 3, 64, seed=3)
    lam, a, b = decays(3), torch.empty((2, 3, 64, 64), device="cuda"), torch.empty((2, 3, 64, 64), device="cuda")
    want = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_out=a)
    q[5, 1], k[140, 1], v[160, 1] = math.nan, math.inf, math.nan
    got = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_out=b)
    clean()
    assert torch.equal(got[:, ::2], want[:, ::2]) and torch.equal(a[:, ::2], b[:, ::2])
    assert bool(got[5, 1].isnan().all()) and torch.equal(got[6:140, 1], want[6:140, 1])
    assert not bool(got[140:150, 1].isfinite().any()) and torch.equal(got[150:160, 1], want[150:160, 1])


@pytest.mark.gpu
def test_linear_packed_bad_bounds(cuda_device):
    q, k, v, gate = linear_inputs(10, 2, 64)
    pool = torch.ones((3, 2, 64, 64), device="cuda")
    fin = torch.full_like(pool, 3.0)
    out = torch.full((10, 2, 64), 7.0, dtype=BF, device="cuda")
    sala.linear_packed_prefill(q, k, v, gate, decays(2), i32([0, 4, 3, 11]), state_in=pool, state_out=fin, out=out)
    torch.cuda.synchronize()
    assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
    assert bool((out[4:] == 7).all()) and bool((fin[1:] == 3).all())
    ref, mag, S, A = ref_linear(q, k, v, gate, decays(2), [0, 4], [pool[0]])
    lin_check(out[:4], ref[:4], mag[:4])
    check(fin[0], S[0], 2.0 ** -16 * A[0] + 1e-30)


@pytest.mark.gpu
def test_linear_packed_graphs_with_a_workspace_each(cuda_device):
    lens = [300, 0, 500]
    cu = i32(starts(lens))
    q, k, v, gate = linear_inputs(800, 4, 128, seed=1)
    lam = decays(4)
    pool = torch.randn((3, 4, 128, 128), generator=gen(4), device="cuda")
    d = sala.PackedLinearDesc(800, 3, 3, 4, 128, sala.SALA_BF16, 1.0)
    need = sala.LIB.sala_linear_packed_workspace_size(ctypes.byref(d))
    runs = []
    for _ in range(2):
        ws, out, fin = sala.workspace(need, "cuda"), torch.empty_like(q), torch.empty_like(pool)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sala.linear_packed_prefill(q, k, v, gate, lam, cu, state_in=pool, state_out=fin, out=out, ws=ws)
        runs.append((g, ws, out, fin))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        for (g, *_), s in zip(runs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    fin = torch.empty_like(pool)
    want = sala.linear_packed_prefill(q, k, v, gate, lam, cu, state_in=pool, state_out=fin)
    clean()
    for _, _, o, f in runs:
        assert torch.equal(o, want) and torch.equal(f, fin)
    cu.copy_(i32([0, 128, 800, 800]))
    want = sala.linear_packed_prefill(q, k, v, gate, lam, cu, state_in=pool, state_out=fin)
    runs[0][0].replay()
    clean()
    assert torch.equal(runs[0][2], want) and torch.equal(runs[0][3], fin)


MANY = [(37 * i * i) % 211 for i in range(70)] + [2500, 1, 0]


@pytest.mark.gpu
def test_many_sequences(cuda_device):
    """More sequences than a warp looks at together, a long one that is cut behind them."""
    cu = starts(MANY)
    T, n = cu[-1], len(MANY)
    q, k, v, gate = dense_inputs(T, 4, 2, 128, seed=4)
    out = sala.dense_prefill(q, k, v, gate, i32(cu))
    ref, mag = ref_dense(q, k, v, gate, cu)
    check(out, ref, attn_tol(ref, mag))
    q, k, v, gate = linear_inputs(T, 2, 128, seed=4)
    lam = decays(2)
    pool = torch.randn((n, 2, 128, 128), generator=gen(4), device="cuda")
    fin = torch.empty_like(pool)
    ref, mag, S, A = ref_linear(q, k, v, gate, lam, cu, list(pool))
    out = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool, state_out=fin)
    lin_check(out, ref, mag)
    for i in range(n):
        check(fin[i], S[i], 2.0 ** -16 * A[i] + 1e-30)
    out = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool)      # outputs only
    lin_check(out, ref, mag)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    again = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool, stream=s)
    s.synchronize()
    assert torch.equal(out, again)
    clean()


# ------------------------------------------------------------------------------------------ step

@pytest.mark.gpu
@pytest.mark.parametrize("B,H,d", [(1, 1, 64), (5, 4, 128), (9, 3, 64), (40, 32, 128)])
@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_linear_packed_step(cuda_device, B, H, d, dtype):
    g = gen(B)
    q, k = unit(g, B, H, d), unit(g, B, H, d)
    v, gate = rnd(g, B, H, d).to(dtype), rnd(g, B, H, d).to(dtype)
    lam = decays(H)
    pool = torch.randn((B + 3, H, d, d), generator=g, device="cuda")
    slots = torch.randperm(B + 3, generator=g, device="cuda")[:B].int()
    if B > 4:
        slots[2] = -1
    old = pool.clone()
    out = torch.full((B, H, d), 7.0, dtype=dtype, device="cuda")
    sala.linear_packed_step(q, k, v, gate, lam, pool, slots=slots, scale=0.25, out=out)
    clean()
    live = [i for i, s in enumerate(slots.tolist()) if s >= 0]
    ref, mag, fin, fabs = ref_linear(q[live], k[live], v[live], gate[live], lam, list(range(len(live) + 1)),
                                     [old[slots[i]] for i in live], scale=0.25)
    step = HALF if dtype == BF else 2.0 ** -24
    # a sum of d products and one fp32 update of the state; sigmoid from fast intrinsics (2^-20)
    check(out[live], ref, step * ref.abs() + 2.0 ** -20 * ref.abs() + (d + 4) * 2.0 ** -24 * mag + 1e-30)
    for i, S, A in zip(live, fin, fabs):
        check(pool[slots[i]], S, 2.0 ** -23 * A + 1e-30)
    for i in range(B):
        if i not in live:
            assert bool((out[i] == 7).all())
    used = set(slots.tolist())
    assert all(torch.equal(pool[p], old[p]) for p in range(B + 3) if p not in used)


@pytest.mark.gpu
def test_linear_packed_step_doubled_slots(cuda_device):
    g = gen(1)
    q, k, v, gate = linear_inputs(4, 2, 64, seed=1)
    pool = torch.randn((2, 2, 64, 64), generator=g, device="cuda")
    solo = pool.clone()
    sala.linear_packed_step(q, k, v, gate, decays(2), solo, slots=i32([1, -1, -1, 0]))
    clean()
    out = torch.full((4, 2, 64), 7.0, dtype=BF, device="cuda")
    sala.linear_packed_step(q, k, v, gate, decays(2), pool, slots=i32([1, 1, 9, 0]), out=out)
    torch.cuda.synchronize()
    assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
    assert torch.equal(pool, solo) and bool((out[1:3] == 7).all())


# ---------------------------------------------------------------------------------------- prefix

PREFIX = [(1, 0, 1, 1, 1, 64), (5, 70, 48, 4, 1, 64), (3, 128, 300, 6, 2, 128), (9, 1000, 700, 16, 1, 128),
          (130, 257, 20, 3, 3, 64), (2, 2000, 64, 128, 1, 128), (4, 0, 513, 32, 8, 128), (3, 1, 1300, 7, 1, 64),
          (6, 640, 130, 100, 1, 64), (40, 1500, 64, 8, 2, 128), (20, 5000, 33, 7, 1, 64), (33, 1025, 200, 24, 3, 128)]


def prefix_inputs(B, P, cap, Hq, Hkv, d, n_slots, seed=0):
    g = gen(seed)
    t = dict(q=unit(g, B, Hq, d), k=unit(g, B, Hkv, d), v=rnd(g, B, Hkv, d), gate=rnd(g, B, Hq, d),
             pk=unit(g, P, Hkv, d) if P else None, pv=rnd(g, P, Hkv, d) if P else None,
             kc=unit(g, n_slots, cap, Hkv, d), vc=rnd(g, n_slots, cap, Hkv, d))
    lens = [(37 * i * i + 11 * i) % cap for i in range(B)]
    lens[0] = cap - 1
    t["lens"] = lens
    t["slots"] = torch.randperm(n_slots, generator=g, device="cuda")[:B].tolist()
    return t


def call_prefix(t, **kw):
    return sala.prefix_decode(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], i32(t["lens"]),
                              slots=i32(t["slots"]), **kw)


@pytest.mark.gpu
@pytest.mark.parametrize("B,P,cap,Hq,Hkv,d", PREFIX)
def test_prefix_decode(cuda_device, B, P, cap, Hq, Hkv, d):
    t = prefix_inputs(B, P, cap, Hq, Hkv, d, B + 2, seed=B + P)
    # what lies at and behind a request's length may be anything
    for s, n in zip(t["slots"], t["lens"]):
        t["kc"][s, n:], t["vc"][s, n:] = math.nan, math.inf
    kc0, vc0 = t["kc"].clone(), t["vc"].clone()
    ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], kc0, vc0, t["lens"], t["slots"])
    out = call_prefix(t)
    clean()
    check(out, ref, attn_tol(ref, mag))
    for b, (s, n) in enumerate(zip(t["slots"], t["lens"])):
        kc0[s, n], vc0[s, n] = t["k"][b], t["v"][b]
    assert torch.equal(t["kc"].view(torch.int16), kc0.view(torch.int16))
    assert torch.equal(t["vc"].view(torch.int16), vc0.view(torch.int16))


@pytest.mark.gpu
def test_prefix_decode_skipped_rows(cuda_device):
    t = prefix_inputs(6, 200, 64, 4, 2, 64, 6, seed=3)
    t["slots"] = [5, -1, 5, 9, 2, 0]
    t["lens"] = [10, 3, 4, 5, 64, 63]
    kc0, vc0 = t["kc"].clone(), t["vc"].clone()
    out = torch.full((6, 4, 64), 7.0, dtype=BF, device="cuda")
    call_prefix(t, out=out)
    torch.cuda.synchronize()
    assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
    ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], kc0, vc0, t["lens"],
                          [5, -1, -1, -1, -1, 0])
    for b in (0, 5):
        check(out[b], ref[b], attn_tol(ref, mag)[b])
    assert bool((out[1:5] == 7).all())
    kc0[5, 10], kc0[0, 63] = t["k"][0], t["k"][5]
    vc0[5, 10], vc0[0, 63] = t["v"][0], t["v"][5]
    assert torch.equal(t["kc"], kc0) and torch.equal(t["vc"], vc0)


@pytest.mark.gpu
def test_prefix_decode_isolation(cuda_device):
    t = prefix_inputs(4, 300, 200, 8, 2, 128, 4, seed=3)
    t["lens"] = [150, 199, 20, 130]
    keep = {n: t[n].clone() for n in ("kc", "vc")}
    want = call_prefix(t)
    for n in keep:
        t[n].copy_(keep[n])
    s = t["slots"][1]
    t["kc"][s, 7, 0, 3] = math.nan
    t["vc"][s, 9, 1, 4] = math.inf
    t["q"][2, 5] = math.inf
    got = call_prefix(t)
    clean()
    ok = torch.ones_like(want, dtype=torch.bool)
    ok[1, :4] = False
    ok[1, 4:, 4] = False
    ok[2, 5] = False
    assert torch.equal(got[ok], want[ok])
    assert bool(got[1, :4].isnan().all()) and bool(got[2, 5].isnan().all()) and not bool(got[1, 4:, 4].isfinite().any())


@pytest.mark.gpu
@pytest.mark.parametrize("P", [500, 12000])
def test_prefix_decode_graph_follows_lengths(cuda_device, P):
    t = prefix_inputs(5, P, 300, 8, 1, 128, 5, seed=8)
    lens, slots = i32([10, 0, 299, 130, 1]), i32(t["slots"])
    out = torch.empty_like(t["q"])
    g = torch.cuda.CUDAGraph()
    call = lambda o: sala.prefix_decode(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], lens,
                                        slots=slots, out=o)
    call(out)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call(out)
    for new in ([10, 0, 299, 130, 1], [255, 128, 3, 0, 299], [0, 0, 0, 0, 0]):
        lens.copy_(i32(new))
        g.replay()
        clean()
        ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], new, t["slots"])
        check(out, ref, attn_tol(ref, mag))
        assert torch.equal(call(None), out)          # the same call gives the same bits


@pytest.mark.gpu
def test_prefix_decode_without_slots_and_on_a_stream(cuda_device):
    t = prefix_inputs(5, 300, 100, 8, 2, 64, 7, seed=2)
    t["slots"] = list(range(5))
    ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], t["lens"], t["slots"])
    lens, s = i32(t["lens"]), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = sala.prefix_decode(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], lens, stream=s)
    s.synchronize()
    check(out, ref, attn_tol(ref, mag))
    clean()


@pytest.mark.gpu
def test_prefix_decode_far_cache_rows(cuda_device):
    """Cache entries whose elements lie beyond 2^32: offsets are 64-bit."""
    cap, Hkv, d, n_slots = 1 << 21, 8, 128, 3
    g = gen(2)
    kc = torch.empty((n_slots, cap, Hkv, d), dtype=BF, device="cuda")
    vc = torch.empty_like(kc)
    n = 300
    kc[2, :n], vc[2, :n] = unit(g, n, Hkv, d), rnd(g, n, Hkv, d)
    kc[0, :n], vc[0, :n] = unit(g, n, Hkv, d), rnd(g, n, Hkv, d)
    q, k, v, gate = dense_inputs(2, 16, Hkv, d, seed=2)
    ref, mag = ref_prefix(q, k, v, gate, None, None, kc, vc, [n, n], [2, 0])
    out = sala.prefix_decode(q, k, v, gate, None, None, kc, vc, i32([n, n]), slots=i32([2, 0]))
    clean()
    check(out, ref, attn_tol(ref, mag))
    assert torch.equal(kc[2, n], k[0]) and torch.equal(vc[0, n], v[1])


# --------------------------------------------------------------------------- a run of them together

@pytest.mark.gpu
@pytest.mark.parametrize("d,H,Hq,Hkv", [(64, 4, 4, 1), (128, 8, 8, 2)])
def test_serving_run(cuda_device, d, H, Hq, Hkv):
    """Prompts behind a shared prefix through a linear and a sparse layer, then decode tokens one by one:
    what the calls give is what one packed prefill over the whole texts gives."""
    P, lens, steps = 200, [30, 1, 129], 4
    n = len(lens)
    full = [P + L + steps for L in lens]
    cu = starts(full)
    T = cu[-1]
    g = gen(11)
    w = [1 + 0.1 * torch.randn((d,), generator=g, device="cuda") for _ in range(4)]
    lam = decays(H)
    lq, lk, lv, lg = rnd(g, T, H, d), rnd(g, T, H, d), rnd(g, T, H, d), rnd(g, T, H, d)
    sq, sk, sv, sg = rnd(g, T, Hq, d), rnd(g, T, Hkv, d), rnd(g, T, Hkv, d), rnd(g, T, Hq, d)
    for t in (lq, lk, lv, lg, sq, sk, sv, sg):           # the texts share their first P tokens
        for i in range(1, n):
            t[cu[i]:cu[i] + P] = t[:P]
    pos = torch.cat([torch.arange(m, device="cuda") for m in full]).int()
    qn, kn = sala.qk_norm(lq, lk, w[0], w[1], pos)
    ref_lin, mag_lin, fin, fabs = ref_linear(qn, kn, lv, lg, lam, cu, [None] * n)
    sqn, skn = sala.qk_norm(sq, sk, w[2], w[3])
    ref_sp, mag_sp = ref_dense(sqn, skn, sv, sg, cu)
    whole_sp = sala.dense_prefill(sqn, skn, sv, sg, i32(cu))
    check(whole_sp, ref_sp, attn_tol(ref_sp, mag_sp))

    # linear layer: prompts without their last tokens, then single tokens
    rows = torch.cat([torch.arange(cu[i], cu[i + 1] - steps, device="cuda") for i in range(n)])
    pool = torch.zeros((n, H, d, d), device="cuda")
    slots = i32([2, 0, 1])
    cu_p = starts([m - steps for m in full])
    out = sala.linear_packed_prefill(qn[rows], kn[rows], lv[rows], lg[rows], lam, i32(cu_p), slots=slots,
                                     state_out=pool)
    clean()
    lin_check(out, ref_lin[rows], mag_lin[rows])
    # sparse layer: caches behind the prefix
    cap = max(lens) + steps
    kc = torch.zeros((n, cap, Hkv, d), dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    for i, s in enumerate([2, 0, 1]):
        kc[s, :lens[i]], vc[s, :lens[i]] = skn[cu[i] + P:cu[i] + P + lens[i]], sv[cu[i] + P:cu[i] + P + lens[i]]
    have = i32(lens)
    pk, pv = skn[:P].contiguous(), sv[:P].contiguous()
    for j in range(steps):
        at = torch.tensor([cu[i + 1] - steps + j for i in range(n)], device="cuda")
        # single tokens through the norm give the bits the packed call gave
        a, b = sala.qk_norm(lq[at], lk[at], w[0], w[1], pos[at])
        assert torch.equal(a, qn[at]) and torch.equal(b, kn[at])
        o = sala.linear_packed_step(a, b, lv[at], lg[at], lam, pool, slots=slots)
        lin_check(o, ref_lin[at], mag_lin[at])
        o = sala.prefix_decode(sqn[at], skn[at], sv[at], sg[at], pk, pv, kc, vc, have, slots=slots)
        check(o, ref_sp[at], attn_tol(ref_sp[at], mag_sp[at]))
        have += 1
    clean()
    for i, s in enumerate([2, 0, 1]):
        check(pool[s], fin[i], 2.0 ** -16 * fabs[i] + 1e-30)


# ------------------------------------------------------------------------- bounds that go back

def usable(cu, T):
    """Sequences that a call computes: usable bounds, and no start below the end of an earlier usable one."""
    top, good = 0, []
    for i, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        if 0 <= a <= b <= T:
            if a >= top:
                good.append(i)
            top = max(top, b)
    return good


# 2500 tokens of two heads of 128 are cut into segments
BACK = [[0, 2500, 0, 2500], [0, 2500, 0, 2500, 0, 2500], [0, 1100, 500, 2500], [2000, 1000, 1000, 2500],
        [0, 9999, 40, 2500], [7, 7, 3, 1200, 1200], list(range(0, 1201, 30)) + [600, 1500, 2500, 100, 200]]


def test_usable_sequences_are_disjoint():
    for cu in BACK:
        good = usable(cu, 2500)
        assert 1 <= len(good) < len(cu) - 1
        assert all(cu[i + 1] <= cu[j] for i, j in zip(good[:-1], good[1:]))


@pytest.mark.gpu
@pytest.mark.parametrize("cu", BACK)
def test_linear_packed_bounds_that_go_back(cuda_device, cu):
    """Sequences that overlap an earlier one are skipped, and the workspace is kept to."""
    T, H, d, n = 2500, 2, 128, len(cu) - 1
    q, k, v, gate = linear_inputs(T, H, d, seed=7)
    lam = decays(H)
    pool = torch.randn((n, H, d, d), generator=gen(4), device="cuda")
    fin = torch.full_like(pool, 3.0)
    out = torch.full((T, H, d), 7.0, dtype=BF, device="cuda")
    desc = sala.PackedLinearDesc(T, n, n, H, d, sala.SALA_BF16, 1.0)
    need = sala.LIB.sala_linear_packed_workspace_size(ctypes.byref(desc))
    assert need > 0
    guard = 64 * H * d * d * 4
    ws = torch.full((need + guard,), 0x5a, dtype=torch.uint8, device="cuda")
    sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu), state_in=pool, state_out=fin, out=out, ws=ws)
    torch.cuda.synchronize()
    assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
    assert sala.sala_get_device_status() == sala.SALA_OK
    assert bool((ws[need:] == 0x5a).all())
    untouched = torch.ones(T, dtype=torch.bool, device="cuda")
    for i in usable(cu, T):
        a, b = cu[i], cu[i + 1]
        untouched[a:b] = False
        ref, mag, S, A = ref_linear(q, k, v, gate, lam, [a, b], [pool[i]])
        if b > a:
            lin_check(out[a:b], ref[a:b], mag[a:b])
        check(fin[i], S[0], 2.0 ** -16 * A[0] + 1e-30)
    assert bool((out[untouched] == 7).all())
    skipped = [i for i in range(n) if i not in usable(cu, T)]
    assert bool((fin[skipped] == 3).all())


@pytest.mark.gpu
@pytest.mark.parametrize("cu", BACK)
def test_dense_bounds_that_go_back(cuda_device, cu):
    T, d = 2500, 64
    q, k, v, gate = dense_inputs(T, 2, 1, d, seed=7)
    out = torch.full((T, 2, d), 7.0, dtype=BF, device="cuda")
    sala.dense_prefill(q, k, v, gate, i32(cu), out=out)
    torch.cuda.synchronize()
    assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
    untouched = torch.ones(T, dtype=torch.bool, device="cuda")
    for i in usable(cu, T):
        a, b = cu[i], cu[i + 1]
        untouched[a:b] = False
        ref, mag = ref_dense(q, k, v, gate, [a, b])
        check(out[a:b], ref[a:b], attn_tol(ref, mag)[a:b])
    assert bool((out[untouched] == 7).all())


# ------------------------------------------------------------------------------------ closed gates

def closed(g, *shape):
    """Gates from wide open to closed: sigmoids of 1 down to 2^-86."""
    return (torch.rand(shape, generator=g, device="cuda") * 70 - 60).to(BF)


# a sigmoid's exponent |gate| log2(e) < 87 is rounded to fp32 (87 2^-24 ln 2 < 2^-18) before an exponential and a
# reciprocal of a few ulp
GATE = 2.0 ** -17


@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,d", [([1], 1, 64), ([130, 1, 300], 4, 128), ([200, 77], 3, 64), ([2500], 2, 128)])
def test_linear_packed_closed_gates(cuda_device, lens, H, d):
    """Positive q, k and v: no sum cancels, so every output has a relative bound, however small its gate."""
    cu, T = starts(lens), sum(lens)
    q, k, v = (x.abs() for x in linear_inputs(T, H, d, seed=T)[:3])
    gate = closed(gen(T + 1), T, H, d)
    lam = decays(H)
    out = sala.linear_packed_prefill(q, k, v, gate, lam, i32(cu))
    clean()
    ref, mag, _, _ = ref_linear(q, k, v, gate, lam, cu, [None] * len(lens))
    check(out, ref, (HALF + GATE) * ref.abs() + HALF * (1 + HALF) * mag + 1e-30)
    # the first token of each sequence through the step: no products in bf16, d fp32 additions (2^-17 for d = 128)
    first = torch.tensor([c for c, n in zip(cu, lens) if n], device="cuda")
    pool = torch.zeros((len(first), H, d, d), device="cuda")
    one = sala.linear_packed_step(q[first], k[first], v[first], gate[first], lam, pool)
    clean()
    check(one, ref[first], (HALF + 3 * GATE) * ref[first].abs() + 1e-30)


@pytest.mark.gpu
def test_dense_and_prefix_closed_gates(cuda_device):
    T, Hq, Hkv, d = 300, 8, 2, 128
    q, k, v, _ = dense_inputs(T, Hq, Hkv, d, seed=5)
    v, gate = v.abs(), closed(gen(6), T, Hq, d)
    out = sala.dense_prefill(q, k, v, gate, i32([0, T]))
    clean()
    ref, mag = ref_dense(q, k, v, gate, [0, T])
    check(out, ref, attn_tol(ref, mag) + GATE * ref)
    t = prefix_inputs(5, 300, 100, Hq, Hkv, d, 7, seed=2)
    t["v"], t["pv"], t["vc"], t["gate"] = t["v"].abs(), t["pv"].abs(), t["vc"].abs(), gate[:5].contiguous()
    ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], t["lens"], t["slots"])
    out = call_prefix(t)
    clean()
    check(out, ref, attn_tol(ref, mag) + GATE * ref)


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("d", [64, 128])
def test_linear_packed_nonfinite_values_keep_no_sign(cuda_device, bad, d):
    """An infinite value leaves infinities of both signs in its column of the state, and q times those is
    NaN: the outputs that see it are NaN in its own tile, as in the tiles behind it and in the step."""
    T, H, u = 300, 2, 40
    q, k, v, gate = linear_inputs(T, H, d, seed=4)
    lam = decays(H)
    want = sala.linear_packed_prefill(q, k, v, gate, lam, i32([0, T]))
    v[u, 1, 9] = bad
    ref, _, S, _ = ref_linear(q, k, v, gate, lam, [0, T], [None])
    assert bool(ref[u:, 1, 9].isnan().all())
    got = sala.linear_packed_prefill(q, k, v, gate, lam, i32([0, T]))
    clean()
    assert bool(got[u:, 1, 9].isnan().all())
    keep = torch.ones_like(want, dtype=torch.bool)
    keep[u:, 1, 9] = False
    assert torch.equal(got[keep], want[keep])
    one = sala.linear_packed_step(*(x[u:u + 1].contiguous() for x in (q, k, v, gate)), lam,
                                  torch.zeros((1, H, d, d), device="cuda"))
    clean()
    assert bool(one[0, 1, 9].isnan())


# ------------------------------------------------------------------ which way a prefix is read

def prefix_need(B, P, cap, Hq, Hkv, d, n_slots=None):
    """Workspace of a prefix decode: none where the prefix is walked with the own keys."""
    return sala.LIB.sala_prefix_workspace_size(ctypes.byref(prefix_desc(
        batch=B, prefix_len=P, n_slots=n_slots or B, q_heads=Hq, kv_heads=Hkv, head_dim=d, cache_capacity=cap)))


def test_a_long_prefix_of_few_requests_is_not_walked():
    """One request has eight CTAs to walk a prefix with: long ones are shared out over the card instead."""
    for Hq, Hkv, d in ((16, 1, 128), (32, 2, 128), (4, 1, 64)):
        for B in (1, 2):
            assert prefix_need(B, 32768, 256, Hq, Hkv, d) > 0
            assert prefix_need(B, 20000, 256, Hq, Hkv, d) > 0
            assert prefix_need(B, 8000, 256, Hq, Hkv, d) == 0
    assert prefix_need(5, 700, 192, 4, 1, 64) == 0 and prefix_need(64, 32768, 1024, 32, 2, 128) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("B,P,cap,Hq,Hkv,d", [(1, 20000, 100, 16, 1, 128), (2, 9300, 700, 8, 2, 64), (1, 9200, 5, 7, 1, 128)])
def test_prefix_decode_of_few_requests(cuda_device, B, P, cap, Hq, Hkv, d):
    t = prefix_inputs(B, P, cap, Hq, Hkv, d, B + 2, seed=B + P)
    ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], t["lens"], t["slots"])
    out = call_prefix(t)
    clean()
    check(out, ref, attn_tol(ref, mag))


def test_a_cache_beyond_64_bits_is_refused():
    for cap, n in ((1 << 62, 4), (1 << 61, 8), ((1 << 63) - 1, 2), (1 << 30, 4)):
        d = prefix_desc(batch=2, prefix_len=32768, n_slots=n, cache_capacity=cap)
        assert sala.LIB.sala_prefix_workspace_size(ctypes.byref(d)) == 0
        assert raw("sala_prefix_decode", d, *[FAKE] * 9, None, FAKE, None, 0) == sala.SALA_ERR_UNSUPPORTED
    d = prefix_desc(batch=2, prefix_len=32768, n_slots=2, cache_capacity=(1 << 30) - 1)
    assert raw("sala_prefix_decode", d, *[FAKE] * 9, None, FAKE, None, 0) == sala.SALA_ERR_WORKSPACE


# --------------------------------------------------------------- slices of per-request arrays

def test_arrays_read_by_value_need_four_byte_alignment():
    """A scheduler hands over slices: 4-byte alignment passes on to the next check (the workspace's)."""
    by4, by2 = ctypes.c_void_p(0x10004), ctypes.c_void_p(0x10002)
    d = lin_desc(tokens=9000, n_seqs=3, heads=32, head_dim=128)
    call = lambda lam, cu, slots: raw("sala_linear_packed_prefill", d, *[FAKE] * 4, lam, cu, slots, None, None, FAKE,
                                      None, 0)
    assert call(by4, by4, by4) == sala.SALA_ERR_WORKSPACE
    for at in range(3):
        assert call(*[by2 if i == at else FAKE for i in range(3)]) == sala.SALA_ERR_INVALID_ARG
    d2 = prefix_desc(prefix_len=32768)
    call = lambda lens, slots: raw("sala_prefix_decode", d2, *[FAKE] * 8, lens, slots, FAKE, None, 0)
    assert call(by4, by4) == sala.SALA_ERR_WORKSPACE
    assert call(by2, FAKE) == call(FAKE, by2) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_qk_norm", qk_desc(), *[FAKE] * 4, by2, FAKE, FAKE) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_dense_prefill", dense_desc(), *[FAKE] * 4, by2, FAKE, FAKE, BIG) == sala.SALA_ERR_INVALID_ARG
    assert raw("sala_linear_packed_step", lin_desc(), *[FAKE] * 4, by2, FAKE, FAKE, FAKE) == sala.SALA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("skip", [1, 2, 3])
def test_slices_of_per_request_arrays(cuda_device, skip):
    tail = lambda x: torch.cat([torch.full((skip,), 99, dtype=x.dtype, device="cuda"), x])[skip:]
    g, cu = gen(3), i32([0, 70, 200, 201])
    w = torch.ones(64, device="cuda")
    q, k, v, gate = linear_inputs(201, 3, 64, seed=3)
    pos = torch.arange(201, device="cuda").int()
    for a, b in zip(sala.qk_norm(q, k, w, w, pos), sala.qk_norm(q, k, w, w, tail(pos))):
        assert torch.equal(a, b)
    assert torch.equal(sala.dense_prefill(q, k, v, gate, cu), sala.dense_prefill(q, k, v, gate, tail(cu)))
    pool, lam, slots = torch.randn((5, 3, 64, 64), generator=g, device="cuda"), decays(3), i32([4, 0, 2])
    one, two = pool.clone(), pool.clone()
    a = sala.linear_packed_prefill(q, k, v, gate, lam, cu, slots=slots, state_in=one, state_out=one)
    b = sala.linear_packed_prefill(q, k, v, gate, tail(lam), tail(cu), slots=tail(slots), state_in=two, state_out=two)
    assert torch.equal(a, b) and torch.equal(one, two)
    a = sala.linear_packed_step(q[:3], k[:3], v[:3], gate[:3], lam, one, slots=slots)
    b = sala.linear_packed_step(q[:3], k[:3], v[:3], gate[:3], tail(lam), two, slots=tail(slots))
    assert torch.equal(a, b) and torch.equal(one, two)
    t = prefix_inputs(3, 500, 100, 8, 2, 64, 5, seed=4)
    lens, slots = i32(t["lens"]), i32(t["slots"])
    call = lambda n, s: sala.prefix_decode(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], n, slots=s)
    assert torch.equal(call(lens, slots), call(tail(lens), tail(slots)))
    clean()


# ---------------------------------------------------------------------------- the Python module

def test_the_older_calls_work_without_the_packed_module():
    """_packed.so belongs to one torch and one Python; where it does not load, only the packed calls fail."""
    code = ("import sys\n"
            "sys.modules['hybrid_sparse_linear_lightning_b200._packed'] = None\n"
            "import torch\n"
            "from hybrid_sparse_linear_lightning_b200 import sala\n"
            "assert sala.sala_version() >= 100 and sala.status_string(0)\n"
            "x = torch.zeros((1, 1, 64), dtype=torch.bfloat16)\n"
            "w = torch.ones(64)\n"
            "try:\n"
            "    sala.qk_norm(x, x, w, w)\n"
            "except ImportError as e:\n"
            "    assert 'build' in str(e)\n"
            "else:\n"
            "    raise SystemExit('the packed call ran')\n")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_another_torch_or_python_needs_a_build(tmp_path, monkeypatch):
    from hybrid_sparse_linear_lightning_b200 import build as B
    for f in ("LIB", "CALLS", "REPORT"):
        monkeypatch.setattr(B, f, str(tmp_path / f))
    assert B.needs_build()
    for f in ("LIB", "CALLS"):
        (tmp_path / f).write_bytes(b"")
    for what, want in ((B.built_for(), False), ({**B.built_for(), "torch": "0"}, True),
                       ({**B.built_for(), "python": "x"}, True), (None, True)):
        (tmp_path / "REPORT").write_text(json.dumps({"registers_per_thread": {}, "built_for": what}))
        assert B.needs_build() is want, what


# ------------------------------------------------- prefixes on both sides of the rule that walks them

def test_workspaces_one_byte_short_are_refused():
    for fn, size, d, n in (("sala_linear_packed_prefill", "sala_linear_packed_workspace_size",
                            lin_desc(tokens=9000, n_seqs=3, heads=32, head_dim=128), 10),
                           ("sala_prefix_decode", "sala_prefix_workspace_size", prefix_desc(prefix_len=32768), 11)):
        need = getattr(sala.LIB, size)(ctypes.byref(d))
        assert need > 0
        assert raw(fn, d, *[FAKE] * n, FAKE, need - 1) == sala.SALA_ERR_WORKSPACE
        assert raw(fn, d, *[FAKE] * n, None, need) == sala.SALA_ERR_WORKSPACE
        assert raw(fn, d, *[FAKE] * n, MISALIGNED, need) == sala.SALA_ERR_INVALID_ARG


@pytest.mark.gpu
@pytest.mark.parametrize("B,P,cap,Hq,Hkv,d", [
    (9, 6000, 700, 16, 1, 128), (2, 3500, 64, 128, 1, 128), (6, 2500, 130, 100, 1, 64), (3, 9000, 100, 17, 1, 128),
    (4, 5000, 33, 66, 2, 64), (1, 10001, 1, 5, 1, 64), (140, 513, 40, 8, 4, 128), (2, 9300, 2000, 128, 2, 128)])
def test_prefix_decode_split(cuda_device, B, P, cap, Hq, Hkv, d):
    """Parts of the prefix joined with the own keys' tiles of 16 heads, for groups of all sizes."""
    assert prefix_need(B, P, cap, Hq, Hkv, d, B + 2) > 0
    test_prefix_decode(cuda_device, B, P, cap, Hq, Hkv, d)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [200, 9000])
def test_prefix_decode_skipped_rows_both_ways(cuda_device, P):
    """Padded, doubled and out-of-range rows leave early, where a second launch waits and where there is none."""
    assert (prefix_need(6, P, 64, 4, 2, 64) > 0) == (P == 9000)
    t = prefix_inputs(6, P, 64, 4, 2, 64, 6, seed=3)
    t["slots"] = [5, -1, 5, 9, 2, 0]
    t["lens"] = [10, 3, 4, 5, 64, 63]
    kc0, vc0 = t["kc"].clone(), t["vc"].clone()
    ref, mag = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], kc0, vc0, t["lens"],
                          [5, -1, -1, -1, -1, 0])
    kc0[5, 10], kc0[0, 63] = t["k"][0], t["k"][5]
    vc0[5, 10], vc0[0, 63] = t["v"][0], t["v"][5]
    for _ in range(3):           # calls one behind the other: an early exit must not let the next one in
        out = torch.full((6, 4, 64), 7.0, dtype=BF, device="cuda")
        call_prefix(t, out=out)
        torch.cuda.synchronize()
        assert sala.sala_get_device_status() == sala.SALA_ERR_DEVICE_FAULT
        for b in (0, 5):
            check(out[b], ref[b], attn_tol(ref, mag)[b])
        assert bool((out[1:5] == 7).all())
        assert torch.equal(t["kc"], kc0) and torch.equal(t["vc"], vc0)
    t["slots"] = [-1] * 6
    out = torch.full((6, 4, 64), 7.0, dtype=BF, device="cuda")
    call_prefix(t, out=out)
    clean()
    assert bool((out == 7).all()) and torch.equal(t["kc"], kc0) and torch.equal(t["vc"], vc0)


@pytest.mark.gpu
@pytest.mark.parametrize("P", [300, 6000])
def test_prefix_decode_isolation_both_ways(cuda_device, P):
    assert (prefix_need(4, P, 200, 8, 2, 128) > 0) == (P == 6000)
    t = prefix_inputs(4, P, 200, 8, 2, 128, 4, seed=3)
    t["lens"] = [150, 199, 20, 130]
    want = call_prefix(t)
    s = t["slots"][1]
    t["kc"][s, 7, 0, 3] = math.nan
    t["vc"][s, 9, 1, 4] = math.inf
    t["q"][2, 5] = math.inf
    t["gate"][3, 1, 6] = math.nan
    got = call_prefix(t)
    clean()
    ok = torch.ones_like(want, dtype=torch.bool)
    ok[1, :4] = False
    ok[1, 4:, 4] = False
    ok[2, 5] = False
    ok[3, 1, 6] = False
    assert torch.equal(got[ok], want[ok])
    assert bool(got[1, :4].isnan().all()) and bool(got[2, 5].isnan().all()) and not bool(got[1, 4:, 4].isfinite().any())
    assert bool(got[3, 1, 6].isnan())
    # the prefix is everyone's: a bad key there reaches the rows of its kv head, and no others
    t["q"][2, 5] = 1.0
    t["pk"][P // 2, 1, 0] = math.nan
    got = call_prefix(t)
    clean()
    assert bool(got[:, 4:].isnan().all())
    assert torch.equal(got[0, :4], want[0, :4]) and torch.equal(got[2, :4], want[2, :4])


@pytest.mark.gpu
@pytest.mark.parametrize("P", [300, 9500])
def test_prefix_decode_on_streams_both_ways(cuda_device, P):
    """Two calls on two streams at once, a workspace each; without slots."""
    assert (prefix_need(5, P, 100, 8, 2, 64, 7) > 0) == (P == 9500)
    runs = []
    for seed in (2, 3):
        t = prefix_inputs(5, P, 100, 8, 2, 64, 7, seed=seed)
        t["slots"] = list(range(5))
        ref = ref_prefix(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], t["lens"], t["slots"])
        runs.append((t, i32(t["lens"]), ref, torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[sala.prefix_decode(t["q"], t["k"], t["v"], t["gate"], t["pk"], t["pv"], t["kc"], t["vc"], lens, stream=s)
             for t, lens, _, s in runs] for _ in range(4)]
    torch.cuda.synchronize()
    for row in outs:
        for out, first, (_, _, (ref, mag), _) in zip(row, outs[0], runs):
            check(out, ref, attn_tol(ref, mag))
            assert torch.equal(out, first)
    clean()


# ------------------------------------------------------------------------------ helper arguments

def test_outs_may_be_any_pair():
    x, w = torch.zeros((2, 1, 64), dtype=BF), torch.ones(64)
    for outs in ([x, x.clone()], (x, x.clone())):         # gets as far as the device
        with pytest.raises(ValueError, match="CUDA device"):
            sala.qk_norm(x, x, w, w, outs=outs)
    for outs in ([x], (x, x, x), x, 5):
        with pytest.raises((TypeError, ValueError), match="outs"):
            sala.qk_norm(x, x, w, w, outs=outs)


@pytest.mark.gpu
def test_qk_norm_outs_in_a_list(cuda_device):
    g = gen(3)
    q, k, w = rnd(g, 5, 4, 64), rnd(g, 5, 2, 64), torch.ones(64, device="cuda")
    want = sala.qk_norm(q, k, w, w)
    outs = [torch.empty_like(q), torch.empty_like(k)]
    assert sala.qk_norm(q, k, w, w, outs=outs) is outs
    with pytest.raises(ValueError, match="outs"):
        sala.qk_norm(q, k, w, w, outs=[q])
    clean()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


def test_a_stream_of_another_device_is_refused():
    """The call runs on the tensors' device; a stream of another one would be ignored there."""
    class Stream:
        device = torch.device("cuda:1")
    z = lambda *s, dt=BF: torch.zeros(s, dtype=dt)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="stream"):
        sala.dense_prefill(z(4, 2, 64), z(4, 1, 64), z(4, 1, 64), z(4, 2, 64), cu, stream=Stream())
    with pytest.raises(ValueError, match="stream"):
        sala.qk_norm(z(4, 2, 64), z(4, 1, 64), torch.ones(64), torch.ones(64), stream=Stream())


def test_what_is_cut_into_segments():
    need = lambda **kw: sala.LIB.sala_linear_packed_workspace_size(ctypes.byref(lin_desc(**{"n_slots": 64, **kw})))
    for heads, d in ((4, 64), (8, 128), (32, 128)):
        assert need(tokens=1024, n_seqs=1, heads=heads, head_dim=d) > 0
        assert need(tokens=896, n_seqs=1, heads=heads, head_dim=d) == 0        # less than eight tiles
        assert need(tokens=1023, n_seqs=8, heads=heads, head_dim=d) == 0       # less than a tile for each
