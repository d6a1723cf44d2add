"""uw_kv4_attention against softmax attention in 64 bits over the values that
the cache's codes stand for.

Bound on o: its rounding to BF16 (8 significant bits: 2^-8 of the value) plus one
rounding of every probability to BF16 in the product with V (2^-8 of
sum p (|v - z| + |z|), z the middle of a vector's range), plus a tenth of the
latter for the fp32 arithmetic of scores and sums.  Bound on lse: fp32 scores of up to a few tens, 2^-10."""
import numpy as np
import pytest
import torch

from tests import _kv4 as ref

pytestmark = pytest.mark.gpu


def _dev(a):
    a = np.ascontiguousarray(a)
    return torch.from_numpy(a.view(np.int16) if a.dtype == np.uint16 else a).cuda()


def _cache(rng, hk, d, page, lens):
    """Random pages; what lies past a sequence's end holds NaN scales and random codes."""
    table, pool = ref.random_table(rng, lens, page)
    pages = ref.Pages(pool, hk, d, page)
    pages.bytes[:] = rng.integers(0, 256, pages.bytes.shape, np.uint8)
    for par in pages.pars:
        scale = ref.f32(ref.bf16(rng.uniform(0.05, 0.5, par.shape[:-1]))).reshape(par.shape[:-1])
        lo = scale * (-7.5 + rng.standard_normal(par.shape[:-1]))
        par[..., 0], par[..., 1] = ref.bf16(scale), ref.bf16(lo)
    for s, m in enumerate(lens):
        if m % page:
            for par in pages.pars:
                par[table[s, m // page], :, m % page:] = 0x7FC0
    return pages, table


def _run(uw, seed, hq, hk, d, page, new, lens, causal=True, window=0, scale=0.0, max_new=None, strided=False,
         change=None, extra=0, hints=True):
    rng = np.random.default_rng(seed)
    pages, table = _cache(rng, hk, d, page, lens)
    t = int(sum(new))
    qb = ref.bf16(1.5 * rng.standard_normal((t + extra, hq, d)))
    if change is not None:
        change(pages, table, qb)
    tab = _dev(table)
    cache = uw.kv4_cache(_dev(pages.bytes), tab, hk, d, page)
    q = _dev(qb)
    out = _dev(np.full(qb.shape, 0x7FC0, np.uint16))
    if strided:
        big = torch.zeros(t + extra, hq + 3, d + 8, dtype=torch.int16, device="cuda")
        big[:, 1:hq + 1, :d] = q
        q = big[:, 1:hq + 1, :d]
        out = torch.full((t + extra, hq + 1, d + 16), 0x7FC0, dtype=torch.int16, device="cuda")[:, :hq, :d]
    lse = torch.full((t + extra, hq), 7.0, device="cuda")
    ws = torch.empty(uw.kv4_workspace_size(cache, hq), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    start, length = _dev(ref.starts(new)), _dev(np.array(lens, np.int32))
    mn, ml = (max(new, default=0) if max_new is None else max_new, max(lens, default=0)) if hints else (0, 0)
    call = lambda: uw.kv4_attention(cache, start, length, q, out, ws, mn, ml, scale=scale, causal=causal,  # noqa: E731
                                    window=window, lse=lse)
    call()
    first = out.contiguous().clone()
    call()                                          # the workspace is ready for the next call
    assert uw.check_status(ws) == 0
    assert torch.equal(first, out)                  # and the same call gives the same bits
    o = ref.f32(first.cpu().numpy().view(np.uint16)).reshape(qb.shape)
    lse = lse.cpu().numpy()
    sm = scale if scale else 1 / np.sqrt(d)
    o_ref, lse_ref, bound = ref.attention(ref.f32(qb).reshape(qb.shape)[:t], pages, table, new, lens, hk, causal,
                                          window, sm)
    assert np.isnan(o[t:]).all() and np.all(lse[t:] == 7.0)
    o, lse = o[:t], lse[:t]
    fine = np.isfinite(o_ref).all(-1)
    assert np.array_equal(np.isnan(o).any(-1), ~fine)
    err = np.abs(o - o_ref)[fine]
    tol = (2.0 ** -8 * np.abs(o_ref) + 1.1 * 2.0 ** -8 * bound + 1e-30)[fine]
    assert np.all(err <= tol), "worst error over its bound %.3g" % np.max(err / tol)
    empty = np.isneginf(lse_ref)
    assert np.array_equal(np.isneginf(lse), empty) and np.all(o[empty] == 0)
    ok = fine & ~empty
    assert np.all(np.abs(lse - lse_ref)[ok] <= 2.0 ** -10)


SINGLE = [
    # hq, hk, D, page, lens: single tokens, groups of 1, 3, 4, 5, 8, 16 and 71 heads, lengths about tiles and pages
    (8, 8, 128, 16, [1]), (8, 2, 128, 16, [2, 15, 16, 17]), (3, 1, 64, 16, [31, 32, 33]),
    (32, 8, 128, 64, [63, 64, 65, 127, 128, 129]), (5, 1, 128, 32, [257]), (8, 1, 64, 128, [1000, 1, 300]),
    (16, 1, 128, 256, [255, 256, 257]), (71, 1, 64, 16, [500]), (12, 4, 64, 32, [2049]),
    (32, 8, 128, 16, [5000, 3, 1200]), (8, 2, 128, 64, [40001]), (4, 4, 64, 16, [20000, 20001]),
]


@pytest.mark.parametrize("hq,hk,d,page,lens", SINGLE)
def test_single_tokens(uw, hq, hk, d, page, lens):
    _run(uw, hq + page, hq, hk, d, page, [1] * len(lens), lens)


FEW = [
    (8, 2, 128, 16, [5, 1, 0, 8], [5, 100, 7, 1000]), (4, 4, 64, 32, [3, 16, 17], [300, 16, 33]),
    (9, 3, 128, 64, [4] * 6, [4, 5, 63, 64, 65, 999]), (8, 1, 64, 16, [2, 7], [3000, 7]),
]


@pytest.mark.parametrize("hq,hk,d,page,new,lens", FEW)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 20), (True, 1), (False, 40)])
def test_few_tokens(uw, hq, hk, d, page, new, lens, causal, window):
    _run(uw, hq, hq, hk, d, page, new, lens, causal, window)


MANY = [
    (4, 2, 128, 16, [64], [64]), (4, 1, 64, 64, [200], [200]), (8, 8, 128, 32, [129, 31], [129, 500]),
    (6, 2, 128, 128, [300, 1, 0, 257], [300, 1000, 50, 700]), (16, 2, 64, 16, [500], [1300]),
    (5, 1, 128, 256, [777], [777]), (4, 4, 128, 64, [1025], [1025]), (7, 1, 64, 32, [333], [2000]),
]


@pytest.mark.parametrize("hq,hk,d,page,new,lens", MANY)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
def test_many_tokens(uw, hq, hk, d, page, new, lens, causal, window):
    _run(uw, hq + 1, hq, hk, d, page, new, lens, causal, window)


@pytest.mark.parametrize("hq,hk,d,page,new,lens", MANY)
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
def test_many_tokens_of_unknown_bounds(uw, hq, hk, d, page, new, lens, causal, window):
    """The same without bounds, which leaves them to the kernel for many rows however short they are."""
    _run(uw, hq + 1, hq, hk, d, page, new, lens, causal, window, hints=False)


@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("hq,hk,new,lens", [(8, 1, [128], [128]), (8, 1, [129], [131]), (8, 1, [127, 130, 1], [900] * 3),
                                            (32, 8, [64, 3], [64, 64]), (4, 4, [90], [5000])])
def test_rows_about_the_choice_of_kernel(uw, hq, hk, new, lens, hints):
    _run(uw, hq + len(new), hq, hk, 128, 32, new, lens, hints=hints)


@pytest.mark.parametrize("max_new,max_len", [(2 ** 62, 2 ** 62), (2 ** 62, 1), (1, 2 ** 62), (2 ** 31, 2 ** 31)])
def test_absurd_bounds(uw, max_new, max_len):
    rng = np.random.default_rng(3)
    pages, table = _cache(rng, 2, 64, 16, [70, 300])
    q = _dev(ref.bf16(rng.standard_normal((71, 4, 64))))
    cache = uw.kv4_cache(_dev(pages.bytes), _dev(table), 2, 64, 16)
    ws = torch.empty(uw.kv4_workspace_size(cache, 4), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    start, length = _dev(ref.starts([70, 1])), _dev(np.array([70, 300], np.int32))
    want, got = torch.empty_like(q), torch.empty_like(q)
    uw.kv4_attention(cache, start, length, q, want, ws, 70, 300)
    uw.kv4_attention(cache, start, length, q, got, ws, max_new, max_len)
    assert uw.check_status(ws) == 0
    diff = ref.f32(want.cpu().numpy().view(np.uint16)) - ref.f32(got.cpu().numpy().view(np.uint16))
    assert np.abs(diff).max() <= 2.0 ** -5      # values of up to 5, two kernels' roundings


@pytest.mark.parametrize("new,lens", [([5], [3]), ([9, 1], [0, 0]), ([200, 2], [150, 1]), ([1, 300], [0, 40])])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_see_nothing(uw, new, lens, causal):
    """More new tokens than the sequence holds: the first have no key (causal), or none does (length 0)."""
    _run(uw, 3, 8, 2, 128, 16, new, lens, causal)


@pytest.mark.parametrize("new", [1, 3, 150])
def test_strided_rows(uw, new):
    _run(uw, new, 8, 2, 64, 16, [new, new], [new + 40, new], strided=True)


@pytest.mark.parametrize("hints", [True, False])
@pytest.mark.parametrize("max_new", [0, 1, 5, 4096])
def test_bounds_only_choose_the_split(uw, max_new, hints):
    """Wrong or missing upper bounds give right results."""
    _run(uw, 5, 8, 2, 128, 32, [1, 90, 4, 260], [900, 90, 64, 300], max_new=max_new, hints=hints)


def test_many_sequences(uw):
    rng = np.random.default_rng(9)
    new = [int(n) for n in rng.integers(0, 3, 700)]
    lens = [n + int(m) for n, m in zip(new, rng.integers(0, 90, 700))]
    _run(uw, 6, 4, 2, 64, 16, new, lens)


def test_tokens_of_no_sequence_are_left_alone(uw):
    _run(uw, 7, 4, 2, 128, 16, [2, 1], [30, 5], extra=4)
    _run(uw, 7, 4, 2, 128, 16, [200, 1], [230, 5], extra=4)


@pytest.mark.parametrize("new", [4, 300])
def test_masked_keys_may_hold_anything(uw, new):
    """A stored NaN key or value reaches the rows that see it and no other."""
    lens = [new + 50]

    def change(pages, table, qb):
        for which, p in ((0, new + 47), (1, new + 48)):    # seen by the last rows only
            pages.pars[which][table[0, p // 16], 0, p % 16] = 0x7FC0
        pages.pars[1][table[0, 0], 1, 3] = 0x7FC0          # position 3, outside the window of head 1's rows

    _run(uw, 8, 4, 2, 128, 16, [new], lens, window=40, change=change)


@pytest.mark.parametrize("new,window", [(1, 5), (1, 16), (3, 40), (20, 100), (200, 300), (200, 33), (1, 1)])
@pytest.mark.parametrize("page", [16, 64])
@pytest.mark.parametrize("hints", [True, False])
def test_pages_before_the_window_may_be_gone(uw, new, window, page, hints):
    """The table holds no page numbers for what every row's window has left behind."""
    lens = [new + 901, new + 75]

    def change(pages, table, qb):
        for s, m in enumerate(lens):
            gone = max(m - new - window + 1, 0) // page
            # the pages hold NaN, and the numbers are none
            for p in table[s, :gone]:
                for par in pages.pars:
                    par[p] = 0x7FC0
            table[s, :gone] = -1

    _run(uw, 13, 8, 2, 128, page, [new, new], lens, window=window, change=change, hints=hints)


@pytest.mark.parametrize("new", [1, 3, 200])
def test_sharp_and_flat_scores(uw, new):
    """One key far above the others (early, late, in between), and all scores equal."""
    def sharp(pages, table, qb):
        for p in (0, 70, 149 + new):
            pages.pars[0][table[0, p // 64], :, p % 64, 0] = ref.bf16(np.float32(40))
            pages.pars[0][table[0, p // 64], :, p % 64, 1] = ref.bf16(np.float32(-300))

    def flat(pages, table, qb):
        qb[:] = 0

    _run(uw, 12, 8, 2, 128, 64, [new], [150 + new], change=sharp)
    _run(uw, 12, 8, 2, 128, 64, [new], [150 + new], change=flat)
    _run(uw, 12, 8, 2, 64, 64, [new], [150 + new], scale=0.01)
    _run(uw, 12, 8, 2, 64, 64, [new], [150 + new], scale=2.0)


@pytest.mark.parametrize("new", [[1, 3], [5, 2], [200, 77]])
@pytest.mark.parametrize("k_up,v_up", [(20, 0), (-20, 0), (0, 30), (0, -30), (12, -12)])
def test_large_and_small_values(uw, new, k_up, v_up):
    """Keys and values far from 1 (the softmax's scale keeps the scores where they were): exact powers of two."""
    def change(pages, table, qb):
        for par, up in zip(pages.pars, (k_up, v_up)):
            finite = (par & 0x7F80) != 0x7F80
            par[:] = np.where(finite, ref.bf16(ref.f32(par).reshape(par.shape) * 2.0 ** up).reshape(par.shape), par)
    _run(uw, 31, 8, 2, 128, 32, new, [600, 333], scale=128 ** -0.5 * 2.0 ** -k_up, change=change)


def test_bad_pages_are_reported(uw):
    hk, d, page = 2, 64, 16
    pages = torch.zeros(2, hk, page * (d + 8), dtype=torch.uint8, device="cuda")
    q = torch.zeros(200, 4, d, dtype=torch.int16, device="cuda")
    for table, length, new in (([[0, 2]], 20, 1), ([[0, -7]], 20, 1), ([[0, 1]], 40, 1), ([[0, 5]], 20, 200)):
        cache = uw.kv4_cache(pages, _dev(np.array(table, np.int32)), hk, d, page)
        ws = torch.empty(uw.kv4_workspace_size(cache, 4), dtype=torch.uint8, device="cuda")
        uw.workspace_init(ws)
        start, ln = _dev(np.array([0, new], np.int32)), _dev(np.array([length], np.int32))
        uw.kv4_attention(cache, start, ln, q[:new], torch.empty_like(q[:new]), ws, new, length)
        assert uw.check_status(ws) == 4


@pytest.mark.parametrize("new", [2, 200])
def test_pages_past_32_bits(uw, new):
    """The same tokens in a pool's first pages and in pages whose offset is beyond 4 GB."""
    hq, hk, d, page, n_pages, length = 8, 8, 128, 256, 16000, 700
    size = uw.kv4_page_bytes(hk, d, page)
    assert (n_pages - 4) * size > 2 ** 32
    pool = torch.empty(n_pages * size, dtype=torch.uint8, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    qkv = torch.randn(length, hq + 2 * hk, d, generator=gen, device="cuda").bfloat16()
    outs = []
    for first in (0, n_pages - 3):
        table = torch.arange(first, first + 3, dtype=torch.int32, device="cuda")[None]
        cache = uw.kv4_cache(pool, table, hk, d, page)
        ws = torch.empty(uw.kv4_workspace_size(cache, hq), dtype=torch.uint8, device="cuda")
        uw.workspace_init(ws)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hk], qkv[:, hq + hk:]
        span = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, length], [length], [0, new])]
        uw.kv4_append(cache, span[0], span[1], None, k, v, None, None, None, ws)
        ko, vo, out = torch.empty_like(k), torch.empty_like(v), torch.empty_like(q[:new])
        uw.kv4_read(cache, span[0], span[1], ko, vo, ws)
        uw.kv4_attention(cache, span[2], span[1], q[:new], out, ws)  # no bounds: few rows and many by their number
        assert uw.check_status(ws) == 0
        outs.append((ko, vo, out))
    for low, high in zip(*outs):
        assert torch.equal(low, high)
    # half a step of the scale, and the rounding of the value read back
    step = (outs[0][0].float() - qkv[:, hq:hq + hk].float()).abs().amax(-1)
    span = qkv[:, hq:hq + hk].float().aminmax(dim=-1)
    assert (step <= (span.max - span.min) / 30 * 1.01 + 2.0 ** -8 * 5).all()


def test_on_another_stream(uw):
    """All work is enqueued on the stream that is passed."""
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        _run(uw, 13, 8, 2, 128, 16, [1, 40], [900, 40])


@pytest.mark.parametrize("new,length", [(1, 700), (260, 700)])
def test_captured_in_a_graph(uw, new, length):
    """A captured step replays with lengths and inputs changed in place."""
    rng = np.random.default_rng(21)
    pages, table = _cache(rng, 2, 128, 16, [length])
    cache = uw.kv4_cache(_dev(pages.bytes), _dev(table), 2, 128, 16)
    ws = torch.empty(uw.kv4_workspace_size(cache, 8), dtype=torch.uint8, device="cuda")
    uw.workspace_init(ws)
    start, ln = _dev(np.array([0, new], np.int32)), _dev(np.array([length], np.int32))
    q = _dev(ref.bf16(rng.standard_normal((new, 8, 128))))
    out, again = torch.empty_like(q), torch.empty_like(q)
    uw.kv4_attention(cache, start, ln, q, out, ws, new, length)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        uw.kv4_attention(cache, start, ln, q, out, ws, new, length)
    ln.fill_(length - 33)
    q.copy_(_dev(ref.bf16(rng.standard_normal((new, 8, 128)))))
    graph.replay()
    uw.kv4_attention(cache, start, ln, q, again, ws, new, length)
    assert uw.check_status(ws) == 0
    assert torch.equal(out, again)
