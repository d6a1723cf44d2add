"""What the attention kernels round, beyond what test_gpu_kv4_attention.py allows
both of them: values that cancel, so that the output's own rounding hides nothing.

With z the middle of a value's range, o = sum p s (c - 8) + sum p z, and
  few rows   p s is the sum of two BF16: each rest is rounded to 2^-8 of at most
             2^-8 of p s, so 2^-16 of sum p |v - z|;
  many rows  p s is one BF16: 2^-8 of sum p |v - z|, and none of sum p |z|.
Both: scores in fp32 from a product in D / 16 steps of 17 terms each, every one
cut to 2^-23 of the largest, so at most 17 * 2^-23 < 2^-18.9 of
a = scale * sum |q| (s c + |lo|); a probability over the sum of all is off by
twice that, taken as 2^-17 a.  Sums over at most 64 keys (8 steps of 17 terms, 2^-16) and the joins,
exponentials and quotients (a few 2^-22): 2^-15.5.  In all, of sum p (|v - z| + |z|):
2^-15 + 2^-17 a.  And the output's rounding, 2^-8 of it."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref

PAGE = 16


def _problem(seed, hq, hk, d, new, length, middle):
    """Keys at random and queries small, so that probabilities are nearly equal; values in pairs of opposite ones,
    their ranges about +- middle steps of a scale that the pair has in common."""
    rng = np.random.default_rng(seed)
    table, pool = ref.random_table(rng, [length], PAGE)
    pages = ref.Pages(pool, hk, d, PAGE)
    pages.bytes[:] = rng.integers(0, 256, pages.bytes.shape, np.uint8)
    kpar, vpar = pages.pars
    s = ref.f32(ref.bf16(rng.uniform(0.1, 0.3, kpar.shape[:-1]))).reshape(kpar.shape[:-1])
    kpar[..., 0], kpar[..., 1] = ref.bf16(s), ref.bf16(-7.5 * s)
    for j in range(length):
        page, slot = table[0, j // PAGE], j % PAGE
        for h in range(hk):
            if j % 2 == 0:
                code = rng.integers(1, 16, d).astype(np.uint8)
                scale = ref.f32(ref.bf16(rng.uniform(0.1, 0.3, 1)))[0]
            up = middle if j % 2 == 0 else -middle
            # scale * (up - 8) in BF16: scales of few bits keep it exact
            scale = np.float32(np.round(scale * 64) / 64)
            pages.put(1, page, slot, h, code if j % 2 == 0 else 16 - code,
                      ref.bf16(np.array([scale, scale * (up - 8)], np.float32)))
    q = ref.bf16(0.05 * rng.standard_normal((new, hq, d)))
    return pages, table, q


def _reference(pages, table, q, hk, new, length):
    """o in 64 bits; the sums of p |v - z| and p (|v - z| + |z|); a; and for every row its keys' p, s, c - 8 and z."""
    hq, d = q.shape[1:]
    x = ref.f32(q).reshape(q.shape).astype(np.float64)
    o, _, both = ref.attention(x, pages, table, [new], [length], hk, False, 0, d ** -0.5)
    near, rows, a = np.zeros_like(o), [], 0.0
    for h in range(hq):
        (kc, kp), (vc, vp) = (pages.get(w, table[0], length, h // (hq // hk)) for w in (0, 1))
        kp, vp = (ref.f32(p).reshape(-1, 2).astype(np.float64) for p in (kp, vp))
        k = kp[:, 1:] + kc * kp[:, :1]
        score = x[:, h] @ k.T / np.sqrt(d)
        p = np.exp(score - score.max(1, keepdims=True))
        z = vp[:, 1] + 8 * vp[:, 0]
        off = np.abs(vc.astype(np.float64) - 8) * vp[:, :1]
        near[:, h] = p @ off / p.sum(1, keepdims=True)
        a = max(a, (np.abs(x[:, h]) @ (kc * kp[:, :1] + np.abs(kp[:, 1:])).T / np.sqrt(d)).max())
        rows.append((p, vp[:, 0], vc.astype(np.float64) - 8, z))
    return o, near, both, a, rows


def _tolerance(o, near, both, a, few):
    return 2.0 ** -8 * np.abs(o) + (2.0 ** -16 if few else 2.0 ** -8) * near + (2.0 ** -15 + 2.0 ** -17 * a) * both


def _r(x):
    return ref.f32(ref.bf16(x.astype(np.float32))).reshape(x.shape).astype(np.float64)


def _rounded(rows, how):
    """The output with p s (`one` or `two` BF16) or p v's middle too (`middle`) rounded, all else exact."""
    outs = []
    for p, s, c, z in rows:
        ps = p * s
        hi = _r(ps)
        used = hi + _r(ps - hi) if how == "two" else hi
        pz = _r(p * z) if how == "middle" else p * z
        outs.append((used @ c + pz.sum(1, keepdims=True)) / p.sum(1, keepdims=True))
    return np.stack(outs, 1)


FEW = [(4, 1, 128, 1, 2), (4, 2, 64, 2, 8), (8, 1, 128, 1, 2), (5, 1, 64, 3, 4), (16, 2, 128, 2, 2), (32, 8, 128, 1, 64)]
MANY = [(4, 1, 128, 60, 2), (8, 2, 64, 90, 4), (4, 4, 128, 130, 2), (8, 1, 64, 40, 16)]


@pytest.mark.parametrize("case", FEW)
def test_bound_for_few_rows_tells_one_rounding_from_two(case):
    hq, hk, d, new, length = case
    pages, table, q = _problem(1, hq, hk, d, new, length, 0)
    o, near, both, a, rows = _reference(pages, table, q, hk, new, length)
    tol = _tolerance(o, near, both, a, True)
    assert np.all(np.abs(_rounded(rows, "two") - o) <= tol)
    if length <= 4:     # (the roundings of many keys average out)
        assert np.any(np.abs(_rounded(rows, "one") - o) > 2 * tol)


@pytest.mark.parametrize("case", MANY)
def test_bound_for_many_rows_tells_a_rounded_middle(case):
    hq, hk, d, new, length = case
    pages, table, q = _problem(2, hq, hk, d, new, length, 128)
    o, near, both, a, rows = _reference(pages, table, q, hk, new, length)
    tol = _tolerance(o, near, both, a, False)
    assert np.all(np.abs(_rounded(rows, "one") - o) <= tol)
    if length <= 4:
        assert np.any(np.abs(_rounded(rows, "middle") - o) > 2 * tol)


def _run(uw, seed, case, middle, few, hints):
    hq, hk, d, new, length = case
    pages, table, qb = _problem(seed, hq, hk, d, new, length, middle)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x).view(np.int16) if x.dtype == np.uint16 else x).cuda()  # noqa: E731
    cache = uw.kv4_cache(dev(pages.bytes), dev(table), hk, d, PAGE)
    ws = torch.empty(uw.kv4_workspace_size(cache, hq), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    q = dev(qb)
    out = torch.empty_like(q)
    uw.kv4_attention(cache, dev(np.array([0, new], np.int32)), dev(np.array([length], np.int32)), q, out, ws,
                     *((new, length) if hints else (0, 0)), causal=False)
    assert uw.check_status(ws) == 0
    o, near, both, a, _ = _reference(pages, table, qb, hk, new, length)
    err = np.abs(ref.f32(out.cpu().numpy().view(np.uint16)).reshape(o.shape) - o)
    tol = _tolerance(o, near, both, a, few)
    assert np.all(err <= tol), "worst error over its bound %.3g" % np.max(err / tol)


# without bounds up to 32 rows take the kernel for few rows by sixteens, more the other
@pytest.mark.gpu
@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("middle", [0, 8])
@pytest.mark.parametrize("case", FEW)
def test_few_rows(uw, case, middle, hints):
    _run(uw, 1, case, middle, True, hints)


@pytest.mark.gpu
@pytest.mark.parametrize("middle", [0, 128])
@pytest.mark.parametrize("case", MANY)
def test_many_rows(uw, case, middle):
    _run(uw, 2, case, middle, False, False)
