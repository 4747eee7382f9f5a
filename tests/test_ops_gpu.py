"""GPU checks of the serving operators against plain 64-bit implementations.

Tolerances (e = torch.finfo(dtype).eps, a rounding is off by at most e / 2
of the value):
  append   one rounding of a 32-bit rotation whose angle is exact to 2^-23:
           |out - ref| <= e/2 |ref| + 2^-21 r, r the pair's length.
  paged    the output's rounding, plus 2^-11 of sum_j p_j |v_j|: the softmax
           weights' share.  32-bit scores of N(0,1) inputs are off by at most
           d 2^-24 sum |q k| / sqrt(d) < 128 * 6e-8 * 12 ~ 9e-5 absolute, an
           exponential by a few 2^-22; both numerator and denominator carry
           them (2 * 1e-4 < 2^-11).  A weight enters as a 16-bit value plus a
           16-bit remainder, at worst 2^-16.
  prompt   the same, plus e/2 of sum_j p_j |v_j|: each weight is rounded once
           to the dtype before the value product.
  sample   the token is the definition's, computed in 64 bits by sorting.
"""
import math

import numpy as np
import pytest
import torch

from persistent_decode_megakernel_02_b200 import workloads as wl

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def mk():
    from persistent_decode_megakernel_02_b200 import mk
    return mk


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def cu_of(lens):
    return [int(x) for x in np.concatenate([[0], np.cumsum(lens)])]


def make_cache(mk, g, lens, nkv, d, page, dtype, spare=2, extra_cols=1):
    """Pages in no order; unused entries and pages beyond the lengths are NaN."""
    pages = [-(-n // page) for n in lens]
    total = sum(pages) + spare
    perm = torch.randperm(total, generator=g, device="cuda").tolist()
    table = np.full((len(lens), max(max(pages), 1) + extra_cols), perm[-1], np.int32)
    at = 0
    for s, n in enumerate(pages):
        table[s, :n] = perm[at:at + n]
        at += n
    k = torch.randn(total, nkv, page, d, generator=g, device="cuda").to(dtype)
    v = torch.randn(total, nkv, page, d, generator=g, device="cuda").to(dtype)
    for p in perm[at:]:
        k[p], v[p] = NAN, NAN
    for s, n in enumerate(lens):
        if n % page:
            k[table[s, n // page], :, n % page:] = NAN
            v[table[s, n // page], :, n % page:] = INF
    return mk.PagedKV(k, v, torch.from_numpy(table).cuda())


def rotate64(x, pos, theta):
    d = x.shape[-1]
    inv = theta ** (-2.0 * torch.arange(d // 2, dtype=torch.float64, device=x.device) / d)
    a = pos.double()[:, None] * inv
    c, s = a.cos()[:, None], a.sin()[:, None]
    x1, x2 = x.double().chunk(2, -1)
    r = torch.sqrt(x1 * x1 + x2 * x2)
    return torch.cat([x1 * c - x2 * s, x2 * c + x1 * s], -1), torch.cat([r, r], -1)


# ---- append -----------------------------------------------------------------

def append_case(mk, lens, starts, nq, nkv, d, page, dtype, theta=5e5, seed=0, fused=False, behind=0, in_place=False,
                keep_k=True):
    g = gen(seed)
    n, rows = sum(lens), sum(lens) + behind
    ends = [a + m if m else 0 for a, m in zip(starts, lens)]
    cache = make_cache(mk, g, ends, nkv, d, page, dtype, extra_cols=0)
    before_k, before_v = cache.k.clone(), cache.v.clone()
    if fused:       # one buffer [rows][(nq + 2 nkv + 1) heads][d], the operands slices of it
        buf = torch.randn(rows, nq + 2 * nkv + 1, d, generator=g, device="cuda").to(dtype)
        q, k, v = buf[:, :nq], buf[:, nq:nq + nkv], buf[:, nq + nkv:nq + 2 * nkv]
    else:
        q, k, v = (torch.randn(rows, h, d, generator=g, device="cuda").to(dtype) for h in (nq, nkv, nkv))
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    q_out = q if in_place else torch.full((rows, nq, d), 7.0, device="cuda", dtype=dtype)
    k_out = k if in_place else torch.full((rows, nkv, d), 7.0, device="cuda", dtype=dtype) if keep_k else None
    status = ints([0])
    mk.kv_append(cache, q, k, v, ints(cu_of(lens)), ints(starts), theta, q_out, k_out, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    pos = torch.tensor([a + i for a, m in zip(starts, lens) for i in range(m)], device="cuda", dtype=torch.float64)
    e = torch.finfo(dtype).eps
    for x, out in ((q0, q_out), (k0, k_out)):
        if out is None:
            continue
        ref, r = rotate64(x[:n], pos, theta)
        assert ((out[:n].double() - ref).abs() <= e / 2 * ref.abs() + 2.0 ** -21 * r + 1e-7).all()
        assert torch.equal(out[n:], (x if in_place else torch.full_like(out, 7.0))[n:])
    assert torch.equal(v, v0)
    # the cache: the new rows, and nothing else
    want_k, want_v = before_k, before_v
    k_rot, r = rotate64(k0[:n], pos, theta)
    i = 0
    table = cache.page_table.tolist()
    for s, (a, m) in enumerate(zip(starts, lens)):
        for p in range(a, a + m):
            at = (table[s][p // page], slice(None), p % page)
            got = cache.k[at].double()
            assert ((got - k_rot[i]).abs() <= e / 2 * k_rot[i].abs() + 2.0 ** -21 * r[i] + 1e-7).all(), (s, p)
            want_k[at], want_v[at] = cache.k[at], v0[i]
            i += 1
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert same(cache.k, want_k) and same(cache.v, want_v)


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("nq,nkv,d,page", [(32, 8, 64, 16), (8, 8, 128, 64), (7, 1, 128, 7), (6, 2, 64, 1), (2, 1, 64, 24)])
def test_append_ragged(mk, dtype, nq, nkv, d, page):
    append_case(mk, [3, 0, 1, 37, 0, 5], [0, 9, 131, 15, 3, 62], nq, nkv, d, page, dtype, seed=nq)


@pytest.mark.parametrize("kw", [dict(fused=True), dict(fused=True, in_place=True), dict(behind=5), dict(in_place=True, behind=3),
                                dict(keep_k=False)], ids=str)
def test_append_layouts(mk, kw):
    append_case(mk, [4, 1, 0, 9], [5, 0, 8, 30], 4, 2, 64, 16, torch.bfloat16, seed=3, **kw)


@pytest.mark.parametrize("start", [0, 1, 4095, 131071, (1 << 20) - 2])
@pytest.mark.parametrize("theta", [1e4, 5e5])
def test_append_far_positions_keep_their_angles(mk, start, theta):
    # fp16's step is small enough to show an angle that is off by 2^-12
    g = gen(1)
    d, page = 128, 1024
    k = torch.zeros(2, 1, page, d, device="cuda", dtype=torch.float16)
    cache = mk.PagedKV(k, k.clone(), (torch.arange(1025, device="cuda", dtype=torch.int32) % 2)[None].contiguous())
    x = torch.randn(2, 1, d, generator=g, device="cuda").half()
    out, ko = torch.empty_like(x), torch.empty_like(x)
    mk.kv_append(cache, x, x, x, ints([0, 2]), ints([start]), theta, out, ko)
    ref, r = rotate64(x, torch.tensor([start, start + 1], device="cuda"), theta)
    assert ((out.double() - ref).abs() <= 2.0 ** -11 * ref.abs() + 2.0 ** -21 * r + 1e-7).all()
    assert torch.equal(out, ko)


@pytest.mark.parametrize("n", [1, 8, 300])
def test_append_one_token_each(mk, n):
    append_case(mk, [1] * n, [(i * 37) % 90 for i in range(n)], 4, 2, 64, 16, torch.bfloat16, seed=n)


def test_append_many_tokens_and_k_only(mk):
    append_case(mk, [700, 333], [100, 0], 4, 1, 128, 32, torch.float16, seed=4)
    g = gen(2)
    cache = make_cache(mk, g, [20], 2, 64, 16, torch.bfloat16)
    k, v = (torch.randn(20, 2, 64, generator=g, device="cuda").bfloat16() for _ in range(2))
    ko = torch.empty_like(k)
    mk.kv_append(cache, None, k, v, ints([0, 20]), ints([0]), 1e4, None, ko)
    ref, r = rotate64(k, torch.arange(20, device="cuda"), 1e4)
    assert ((ko.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * r + 1e-7).all()


def test_append_bad_values_are_left_out(mk):
    g = gen(5)
    k = torch.zeros(4, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
    # sequence 0: page 9 does not exist; 1: fine; 2: negative start; 3: past the table
    cache = mk.PagedKV(k, k.clone(), ints([[9, 0], [1, 2], [-1, 3], [3, 3]]))
    x = torch.randn(8, 2, 64, generator=g, device="cuda").bfloat16()
    out = torch.full_like(x, 7.0)
    status = ints([0])
    mk.kv_append(cache, x, x, x, ints([0, 2, 4, 6, 8]), ints([0, 3, -1, 31]), 1e4, out, status=status)
    assert int(status) == mk.MK_ERR_INVALID
    bad = [0, 1, 4, 5, 7]          # 5: position 0 of sequence 2 lies on page -1
    assert (out[bad] == 7).all() and not (out[[2, 3, 6]] == 7).all()
    assert torch.equal(cache.v[1, :, 3:5].transpose(0, 1), x[2:4])
    assert torch.equal(cache.v[3, :, 15], x[6])
    cache.v[1, :, 3:5] = 0
    cache.v[3, :, 15] = 0
    assert (cache.v == 0).all()


@pytest.mark.parametrize("cu", [[0, 5, 3, 4, 4], [0, 2, 900, 900, 4], [-3, 1, 2, 3, 4], [2, 3, 3, 4, 4]])
def test_append_broken_offsets_stay_inside(mk, cu):
    # rows no sequence owns, or that lie behind the buffers: nothing out of
    # bounds, what is written lies on a row of the cache
    k = torch.zeros(8, 1, 16, 64, device="cuda", dtype=torch.bfloat16)
    guard = torch.full((8, 1, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    cache = mk.PagedKV(k, k.clone(), ints([[0, 1], [2, 3], [4, 5], [6, 7]]))
    x = torch.ones(4, 1, 64, device="cuda", dtype=torch.bfloat16)
    mk.kv_append(cache, x, x, x, ints(cu), ints([0, 0, 0, 0]), 1e4, guard[:4])
    torch.cuda.synchronize()
    assert (guard[4:] == 7).all()


# ---- paged attention --------------------------------------------------------------

def paged_reference(cache, q, lens, scale):
    n, nq, d = q.shape
    G = nq // cache.n_kv_heads
    out = torch.zeros(n, nq, d, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(out)
    for s, m in enumerate(lens):
        if m == 0:
            continue
        pages = cache.page_table[s, :-(-m // cache.page_size)].long()
        k = cache.k[pages].transpose(0, 1).reshape(cache.n_kv_heads, -1, d)[:, :m].double()
        v = cache.v[pages].transpose(0, 1).reshape(cache.n_kv_heads, -1, d)[:, :m].double()
        w = torch.softmax(q[s].double().view(-1, G, d) @ k.transpose(1, 2) * scale, -1)
        out[s], mass[s] = (w @ v).view(nq, d), (w @ v.abs()).view(nq, d)
    return out, mass


def paged_check(cache, q, lens, out, scale, sel=None):
    ref, mass = paged_reference(cache, q, lens, scale)
    e = torch.finfo(q.dtype).eps
    bad = (out.double() - ref).abs() > e / 2 * ref.abs() + 2.0 ** -11 * mass + 1e-7
    bad |= ~torch.isfinite(out)
    if sel is not None:
        bad = bad[sel]
    assert not bad.any(), (int(bad.sum()), (out.double() - ref).abs().max())


def paged_case(mk, lens, nq, nkv, d, page, dtype, seed=0, max_len=None, scale=None, q_scale=1.0):
    g = gen(seed)
    cache = make_cache(mk, g, lens, nkv, d, page, dtype)
    q = (torch.randn(len(lens), nq, d, generator=g, device="cuda") * q_scale).to(dtype)
    out = torch.full_like(q, NAN)
    status = ints([0])
    mk.paged_attention(cache, q, ints(lens), max(lens) if max_len is None else max_len, out, scale=scale,
                       status=status)
    assert int(status) == 0
    paged_check(cache, q, lens, out, d ** -0.5 if scale is None else scale)
    return cache, q, out


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 64), (32, 8, 128), (1, 1, 64), (8, 1, 128), (6, 2, 64), (14, 2, 128), (3, 1, 128), (10, 2, 64), (8, 8, 64)])
@pytest.mark.parametrize("page", [16, 7])
def test_paged_head_layouts(mk, dtype, nq, nkv, d, page):
    paged_case(mk, [5, 0, 1, 130, 333], nq, nkv, d, page, dtype, seed=nq + d)


@pytest.mark.parametrize("page", [1, 8, 16, 24, 32, 50, 64, 128, 560])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_page_sizes_and_lengths(mk, page, d):
    paged_case(mk, [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 0, 511, 513, 700], 4, 2, d, page,
               torch.bfloat16, seed=page)


@pytest.mark.parametrize("lens,nq,nkv,d,page", [([16385], 32, 8, 64, 64), ([70001], 8, 1, 128, 16), ([1, 30000, 0, 7, 9999], 16, 4, 128, 128),
                                                ([4097] * 40, 32, 8, 64, 32), ([100003], 2, 2, 64, 50)])
def test_paged_long_contexts_split_and_joined(mk, lens, nq, nkv, d, page):
    paged_case(mk, lens, nq, nkv, d, page, torch.float16, seed=len(lens))


def test_paged_many_sequences(mk):
    rng = np.random.default_rng(0)
    paged_case(mk, [int(x) for x in rng.integers(0, 400, 300)], 8, 2, 64, 16, torch.bfloat16)


def test_paged_bound_above_the_lengths_and_sharp_scores(mk):
    # a launch sized for 4096 positions, lengths far below; scores spread over hundreds
    paged_case(mk, [3, 0, 40, 200], 8, 2, 128, 512, torch.float16, max_len=512, seed=1)
    # one-hot softmax: the score error bound scales with |q|, the weights are 0 or 1 beyond it
    g = gen(3)
    cache = make_cache(mk, g, [900], 2, 64, 16, torch.bfloat16)
    q = (torch.randn(1, 8, 64, generator=g, device="cuda") * 64).bfloat16()
    out = torch.empty_like(q)
    mk.paged_attention(cache, q, ints([900]), 900, out)
    ref, mass = paged_reference(cache, q, [900], 0.125)
    # scores up to ~64 sqrt(64) * 5: their 32-bit error is 64 times the one above
    assert ((out.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 64 * 2.0 ** -11 * mass).all()


def test_paged_rising_scores(mk):
    # the running maximum rises at every position, in every split
    g = gen(8)
    n, d, page = 5000, 64, 16
    cache = make_cache(mk, g, [n], 1, d, page, torch.float16)
    q = torch.ones(1, 4, d, device="cuda", dtype=torch.float16)
    table = cache.page_table[0].tolist()
    ramp = (torch.arange(n, device="cuda") / n * 2).half()
    for p in range(-(-n // page)):
        m = min(page, n - p * page)
        cache.k[table[p], 0, :m] = ramp[p * page:p * page + m, None]
    out = torch.empty_like(q)
    mk.paged_attention(cache, q, ints([n]), n, out)
    paged_check(cache, q, [n], out, d ** -0.5)


def test_paged_strides_and_scale(mk):
    g = gen(4)
    cache = make_cache(mk, g, [70, 9, 200], 2, 64, 16, torch.bfloat16)
    big = torch.randn(3, 11, 64, generator=g, device="cuda").bfloat16()
    out = torch.full((3, 9, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    q = big[:, 2:10]
    mk.paged_attention(cache, q, ints([70, 9, 200]), 200, out[:, :8], scale=0.3)
    paged_check(cache, q, [70, 9, 200], out[:, :8], 0.3)
    assert (out[:, 8] == 7).all()


def test_paged_bad_values(mk):
    g = gen(6)
    cache = make_cache(mk, g, [100, 60, 40], 2, 64, 16, torch.bfloat16, spare=0)
    q = torch.randn(3, 4, 64, generator=g, device="cuda").bfloat16()
    out, status = torch.empty_like(q), ints([0])
    # lengths beyond max_len and below zero are clamped
    mk.paged_attention(cache, q, ints([100, 60, -5]), 40, out, status=status)
    assert int(status) == mk.MK_ERR_INVALID
    paged_check(cache, q, [40, 40, 0], out, 0.125)
    # positions on pages that do not exist are left out
    status.zero_()
    good = cache.page_table.clone()
    cache.page_table[0, 1], cache.page_table[0, 6], cache.page_table[1, 0] = -1, 10 ** 6, cache.num_pages
    mk.paged_attention(cache, q, ints([100, 60, 40]), 100, out, status=status)
    assert int(status) == mk.MK_ERR_INVALID
    keep = [p for p in range(100) if p // 16 not in (1, 6)]
    for s, rows in ((0, keep), (1, list(range(16, 60))), (2, list(range(40)))):
        k = cache.k[good[s].long()].transpose(0, 1).reshape(2, -1, 64)[:, rows].double()
        v = cache.v[good[s].long()].transpose(0, 1).reshape(2, -1, 64)[:, rows].double()
        w = torch.softmax(q[s].double().view(2, 2, 64) @ k.transpose(1, 2) * 0.125, -1)
        ref, mass = (w @ v).view(4, 64), (w @ v.abs()).view(4, 64)
        assert ((out[s].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -11 * mass + 1e-7).all(), s


def test_paged_masked_garbage_and_overflowing_scores(mk):
    # an infinity among the keys a row sees: what the formula gives, and only there
    g = gen(7)
    cache = make_cache(mk, g, [50, 50], 1, 64, 16, torch.float16)
    q = torch.ones(2, 2, 64, device="cuda", dtype=torch.float16)
    out = torch.empty_like(q)
    cache.k[cache.page_table[0, 1], 0, 3] = NAN
    mk.paged_attention(cache, q, ints([50, 50]), 50, out)
    assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()
    cache.k[cache.page_table[0, 1], 0, 3] = -INF     # weight zero
    mk.paged_attention(cache, q, ints([50, 50]), 50, out)
    paged_check(cache, q, [50, 50], out, 0.125)


def test_paged_graph_replay_while_lengths_grow(mk):
    g = gen(9)
    full = [900, 40, 300]
    cache = make_cache(mk, g, full, 2, 64, 16, torch.bfloat16)
    q = torch.randn(3, 8, 64, generator=g, device="cuda").bfloat16()
    outs = [torch.empty_like(q) for _ in range(2)]
    lens = ints([1, 1, 1])
    side = torch.cuda.Stream()
    graphs = []
    for o in outs:            # two graphs, each with a workspace of its own
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=side):
            mk.paged_attention(cache, q, lens, 900, o)
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for now in ([1, 0, 5], [200, 40, 299], full):
        lens.copy_(ints(now))
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        for o in outs:
            paged_check(cache, q, now, o, 0.125)


def test_paged_results_repeat_bit_for_bit_on_any_stream(mk):
    g = gen(10)
    lens = [5000, 17, 1200]
    cache = make_cache(mk, g, lens, 4, 128, 32, torch.bfloat16)
    q = torch.randn(3, 16, 128, generator=g, device="cuda").bfloat16()
    first = torch.empty_like(q)
    mk.paged_attention(cache, q, ints(lens), 5000, first)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    l = ints(lens)
    outs = [torch.empty_like(q) for _ in range(6)]
    torch.cuda.synchronize()
    for i, o in enumerate(outs):
        mk.paged_attention(cache, q, l, 5000, o, stream=st if i % 2 else None)
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


def test_paged_workspace_too_small_is_refused(mk):
    g = gen(11)
    cache = make_cache(mk, g, [9000], 1, 64, 16, torch.bfloat16)
    q = torch.randn(1, 8, 64, generator=g, device="cuda").bfloat16()
    ws = mk.paged_attention_workspace(cache, 8, 9000)
    if ws.numel() > 0:
        with pytest.raises(mk.MkError):
            mk.paged_attention(cache, q, ints([9000]), 9000, torch.empty_like(q), workspace=ws[:-16])
    mk.paged_attention(cache, q, ints([9000]), 9000, torch.empty_like(q), workspace=ws)
    torch.cuda.synchronize()


# ---- prompt attention ---------------------------------------------------------------

def prompt_reference(q, k, v, lens, scale):
    n, nq, d = q.shape
    G = nq // k.shape[1]
    out = torch.zeros(n, nq, d, dtype=torch.float64, device="cuda")
    mass = torch.zeros_like(out)
    at = 0
    for m in lens:
        r = slice(at, at + m)
        at += m
        if m == 0:
            continue
        kk = k[r].double().transpose(0, 1).repeat_interleave(G, 0)
        vv = v[r].double().transpose(0, 1).repeat_interleave(G, 0)
        s = q[r].double().transpose(0, 1) @ kk.transpose(1, 2) * scale
        w = torch.softmax(s.masked_fill(torch.ones(m, m, dtype=torch.bool, device="cuda").triu(1), -INF), -1)
        out[r], mass[r] = (w @ vv).transpose(0, 1), (w @ vv.abs()).transpose(0, 1)
    return out, mass


def prompt_check(q, k, v, lens, out, scale):
    ref, mass = prompt_reference(q, k, v, lens, scale)
    e = torch.finfo(q.dtype).eps
    n = sum(lens)
    bad = (out.double() - ref).abs() > e / 2 * ref.abs() + (e / 2 + 2.0 ** -11) * mass + 1e-7
    bad |= ~torch.isfinite(out)
    bad = bad[:n]
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())


def prompt_inputs(lens, nq, nkv, d, dtype, seed=0, behind=0):
    g = gen(seed)
    n = sum(lens) + behind
    return [torch.randn(n, h, d, generator=g, device="cuda").to(dtype) for h in (nq, nkv, nkv)]


def prompt_case(mk, lens, nq, nkv, d, dtype, seed=0, max_len=None):
    q, k, v = prompt_inputs(lens, nq, nkv, d, dtype, seed)
    out, status = torch.full_like(q, NAN), ints([0])
    mk.prompt_attention(q, k, v, ints(cu_of(lens)), max(lens) if max_len is None else max_len, out, status=status)
    assert int(status) == 0
    prompt_check(q, k, v, lens, out, d ** -0.5)


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("nq,nkv,d", [(32, 8, 64), (32, 8, 128), (1, 1, 64), (8, 1, 128), (6, 2, 64), (7, 1, 64), (10, 2, 128), (3, 3, 128)])
def test_prompt_head_layouts(mk, dtype, nq, nkv, d):
    prompt_case(mk, [39, 1, 0, 200, 129], nq, nkv, d, dtype, seed=nq)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 31, 39, 63, 64, 65, 127, 128, 129, 191, 192, 193, 255, 256, 257, 383, 385, 511, 513, 1000, 1025])
def test_prompt_lengths(mk, n, d):
    prompt_case(mk, [n], 4, 2, d, torch.bfloat16, seed=n)


@pytest.mark.parametrize("lens", [[1] * 50, [0, 0, 5, 0], [128, 128, 128], [256, 1, 255, 2, 257], [1500, 3, 700, 0, 64, 2049], [0, 0]])
def test_prompt_packings(mk, lens):
    if sum(lens) == 0:
        q = torch.full((4, 2, 64), 3.0, device="cuda", dtype=torch.float16)
        out = torch.full_like(q, 7.0)
        mk.prompt_attention(q, q, q, ints([0, 0, 0]), 4, out)
        assert (out == 7).all()
        return
    prompt_case(mk, lens, 8, 2, 64, torch.float16, seed=len(lens))
    prompt_case(mk, lens, 4, 4, 128, torch.bfloat16, seed=len(lens), max_len=max(lens) + 77)


def test_prompt_long(mk):
    prompt_case(mk, [5003], 2, 1, 128, torch.bfloat16)
    prompt_case(mk, [4999, 2500], 2, 2, 64, torch.float16)


def test_prompt_rows_behind_and_strides(mk):
    g = gen(2)
    lens = [70, 0, 131]
    n = sum(lens)
    buf = torch.randn(n + 9, 4 + 2 + 2 + 1, 64, generator=g, device="cuda").bfloat16()
    buf[n:] = NAN                    # rows behind the last sequence may hold anything
    out = torch.full((n + 9, 5, 64), 7.0, device="cuda", dtype=torch.bfloat16)
    q, k, v = buf[:, :4], buf[:, 4:6], buf[:, 6:8]
    mk.prompt_attention(q, k, v, ints(cu_of(lens)), 131, out[:, :4], scale=0.2)
    prompt_check(q[:n], k[:n], v[:n], lens, out[:n, :4], 0.2)
    assert (out[n:] == 7).all() and (out[:, 4] == 7).all()


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("what", [NAN, INF, -INF], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("at", [(1, 40), (1, 299), (0, 0), (1, 130)])
def test_prompt_later_tokens_never_reach_a_row(mk, d, what, at):
    # a token whose key and value are NaN or infinite: rows before it and the
    # other sequences are as if it were absent, rows after it as the formula has it
    lens, dtype = [100, 300, 90], torch.bfloat16
    q, k, v = prompt_inputs(lens, 2, 1, d, dtype, seed=5)
    row = cu_of(lens)[at[0]] + at[1]
    end = cu_of(lens)[at[0] + 1]
    clean = torch.empty_like(q)
    mk.prompt_attention(q, k, v, ints(cu_of(lens)), 300, clean)
    out = torch.empty_like(q)
    v2 = v.clone()
    v2[row, 0, 5] = what
    mk.prompt_attention(q, k, v2, ints(cu_of(lens)), 300, out)
    touched = torch.zeros(q.shape, dtype=torch.bool, device="cuda")
    touched[row:end, :, 5] = True
    assert torch.equal(out[~touched], clean[~touched])
    got = out[touched]
    # the weight may underflow to zero, and 0 * inf is NaN as in the plain formula
    assert (torch.isnan(got) | (got == what)).all()
    k2 = k.clone()
    k2[row] = NAN
    mk.prompt_attention(q, k2, v, ints(cu_of(lens)), 300, out)
    touched[row:end] = True
    assert torch.equal(out[~touched], clean[~touched]) and torch.isnan(out[touched]).all()


def test_prompt_sharp_and_rising_scores(mk):
    # the running maximum rises by far more than a rescale bound from tile to tile
    n, d = 700, 64
    q, k, v = prompt_inputs([n], 2, 1, d, torch.float16, seed=9)
    q.fill_(1.0)
    k.copy_((torch.arange(n, device="cuda") / n * 16).half()[:, None, None].expand_as(k))
    out = torch.empty_like(q)
    mk.prompt_attention(q, k, v, ints([0, n]), n, out)
    prompt_check(q, k, v, [n], out, d ** -0.5)
    k.copy_(k.flip(0))               # and falls
    mk.prompt_attention(q, k, v, ints([0, n]), n, out)
    prompt_check(q, k, v, [n], out, d ** -0.5)


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [0, 10, 400, 20], [-4, 10, 15, 20], [0, 10, 15, 50]])
def test_prompt_broken_offsets(mk, cu):
    q, k, v = prompt_inputs([20], 2, 1, 64, torch.bfloat16, behind=10)
    out, status = torch.full_like(q, 7.0), ints([0])
    mk.prompt_attention(q, k, v, ints(cu), 16, out, status=status)
    torch.cuda.synchronize()
    assert int(status) == mk.MK_ERR_INVALID


def test_prompt_longer_than_the_bound_is_left_out(mk):
    lens = [30, 50, 20]
    q, k, v = prompt_inputs(lens, 2, 1, 64, torch.bfloat16)
    out, status = torch.full_like(q, 7.0), ints([0])
    mk.prompt_attention(q, k, v, ints(cu_of(lens)), 40, out, status=status)
    assert int(status) == mk.MK_ERR_INVALID
    ref, _ = prompt_reference(q, k, v, lens, 0.125)
    assert (out[30:80] == 7).all()
    rest = list(range(30)) + list(range(80, 100))
    assert torch.allclose(out[rest].double(), ref[rest], atol=0.05)


def test_prompt_two_streams_and_a_graph(mk):
    lens = [300, 77]
    q, k, v = prompt_inputs(lens, 4, 2, 128, torch.float16)
    cu = ints(cu_of(lens))
    a, b, c = (torch.empty_like(q) for _ in range(3))
    st = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        mk.prompt_attention(q, k, v, cu, 300, c)
    torch.cuda.synchronize()
    mk.prompt_attention(q, k, v, cu, 300, a)
    mk.prompt_attention(q, k, v, cu, 300, b, stream=st)
    gr.replay()
    torch.cuda.synchronize()
    prompt_check(q, k, v, lens, a, 128 ** -0.5)
    assert torch.equal(a, b) and torch.equal(a, c)


# ---- sampling ------------------------------------------------------------------------

def sample_reference(row, t, k, p, m, u):
    """The definition, by sorting, in 64 bits."""
    row = row.astype(np.float64)
    row = np.where(np.isnan(row), -np.inf, row)
    top = row.max()
    if top == -np.inf:
        return -1
    if not t > 0:
        return int(np.argmax(row))
    with np.errstate(invalid="ignore"):
        w = np.where(row == top, 1.0, np.where(np.isinf(row), 0.0, np.exp((row - top) / float(t))))
    if top == np.inf:
        w = (row == top).astype(np.float64)
    order = np.argsort(-row, kind="stable")
    if 0 < k < len(row):
        order = order[:k]
    if p < 1:
        mass = np.cumsum(w[order])
        before = mass - w[order]
        order = order[:max(1, int((before < max(float(p), 0.0) * mass[-1]).sum()))]
    keep = np.zeros(len(row), bool)
    keep[order] = True
    keep &= w >= min(max(float(m), 0.0), 1.0)
    at = np.flatnonzero(keep & (w >= 2.0 ** -43))
    run = np.cumsum(w[at])
    u = min(max(float(u), 0.0), 1.0)
    return int(at[min(int(np.searchsorted(run, u * run[-1], side="right")), len(at) - 1)])


def sample_case(mk, logits, t=None, k=None, p=None, m=None, u=None, seed=0):
    rows = logits.shape[0]
    u = torch.rand(rows, generator=gen(seed), device="cuda") if u is None else u
    f = lambda x: None if x is None else torch.tensor(x, dtype=torch.float32, device="cuda")
    token = torch.full((rows,), -7, dtype=torch.int32, device="cuda")
    mk.sample(logits, u, token, f(t), None if k is None else ints(k), f(p), f(m))
    ln, un = logits.cpu().numpy(), u.cpu().numpy()
    f32 = lambda x, i, off: off if x is None else float(np.float32(x[i]))
    want = [sample_reference(ln[i], f32(t, i, 1.0), 0 if k is None else k[i], f32(p, i, 1.0), f32(m, i, 0.0), un[i])
            for i in range(rows)]
    assert token.tolist() == want


def noise(rows, vocab, seed=0, scale=2.0, ties=False):
    x = torch.randn(rows, vocab, generator=gen(seed), device="cuda") * scale
    return x.bfloat16().float() if ties else x


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("vocab", [1, 2, 31, 33, 1000, 4096, 32003, 128256])
def test_sample_every_filter(mk, vocab, ties):
    rows = 24
    rng = np.random.default_rng(vocab)
    on = [(i & 1, i >> 1 & 1, i >> 2 & 1) for i in range(rows)]
    k = [int(rng.choice([1, 2, 7, 50, 300])) if a else 0 for a, _, _ in on]
    p = [float(rng.choice([0.1, 0.5, 0.9, 0.99])) if b else 1.0 for _, b, _ in on]
    m = [float(rng.choice([0.001, 0.05, 0.5])) if c else 0.0 for _, _, c in on]
    t = [float(x) for x in rng.choice([0.0, 0.3, 0.8, 1.0, 1.7], rows)]
    sample_case(mk, noise(rows, vocab, vocab, ties=ties), t, k, p, m, seed=vocab)


def test_sample_defaults_and_large_vocabulary(mk):
    sample_case(mk, noise(3, 50257))
    sample_case(mk, noise(2, mk.MAX_VOCAB), k=[0, 1000], p=[0.9, 0.95])
    sample_case(mk, noise(1, mk.MAX_VOCAB - 1, ties=True), p=[0.7])


def test_sample_strided_rows(mk):
    buf = noise(6, 1001, 3)
    sample_case(mk, buf[::2, 3:1000], k=[5, 0, 0], p=[1.0, 0.8, 1.0])


def test_sample_equal_logits(mk):
    # every logit the same: top-k and top-p keep the lowest indices
    x = torch.zeros(6, 5000, device="cuda")
    u = torch.tensor([0.0, 0.5, 0.999, 0.25, 0.75, 0.999], device="cuda")
    sample_case(mk, x, k=[10, 10, 10, 0, 0, 4999], p=[1.0, 1.0, 1.0, 0.5, 0.01, 0.5], u=u)
    x[:, 1000:] = -0.0               # equal to +0
    sample_case(mk, x, k=[1500] * 6, u=u)


def test_sample_masked_rows(mk):
    x = noise(8, 3001, 5)
    x[0] = -INF                      # nothing left
    x[1] = NAN
    x[2, :] = -INF
    x[2, 77] = -1e30                 # one left
    x[3, ::2] = -INF
    x[4, 5::7] = NAN
    x[5, 100] = INF
    x[6, [9, 2000]] = INF
    x[7] = torch.finfo(torch.float32).min
    x[7, 3000] = 0.0
    for kw in (dict(), dict(k=[5] * 8), dict(p=[0.9] * 8), dict(m=[0.2] * 8), dict(t=[0.0] * 8),
               dict(k=[3] * 8, p=[0.5] * 8, m=[0.1] * 8), dict(k=[2000] * 8, p=[0.999] * 8)):
        sample_case(mk, x, **kw)


def test_sample_extreme_parameters(mk):
    x = noise(10, 2000, 6)
    tiny = float(np.float32(1e-45))
    sample_case(mk, x, t=[0.0, -1.0, NAN, tiny, 1e-3, 1e3, 3e38, INF, 1.0, 1.0])
    sample_case(mk, x, k=[-1, 0, 1, 2000, 2001, 1999, 1 << 30, 2, 3, -(1 << 31)])
    sample_case(mk, x, p=[0.0, -1.0, 1.0, 2.0, NAN, 1e-9, 0.9999999, INF, -INF, 0.5])
    sample_case(mk, x, m=[0.0, -1.0, 1.0, 2.0, 1e-30, 0.999, INF, 0.5, -INF, 0.1])
    u = torch.tensor([0.0, 1.0, 2.0, -1.0, 0.99999994, 1e-30, 0.5, 0.1, 0.9, 0.3], device="cuda")
    sample_case(mk, x, u=u)
    sample_case(mk, x, k=[3] * 10, u=u)


def test_sample_follows_its_distribution(mk):
    # frequencies over evenly spread uniforms are the probabilities
    n, v = 4096, 50
    row = noise(1, v, 7, scale=1.0)
    u = (torch.arange(n, device="cuda") + 0.5) / n
    token = torch.empty(n, dtype=torch.int32, device="cuda")
    mk.sample(row.expand(n, v).contiguous(), u, token)
    got = torch.bincount(token.long(), minlength=v).double() / n
    assert (got - torch.softmax(row[0].double(), 0)).abs().max() <= 1.0 / n + 1e-9


def test_sample_in_a_graph_and_on_streams(mk):
    x = noise(4, 128256, 8)
    u = torch.rand(4, generator=gen(1), device="cuda")
    k, p = ints([50] * 4), torch.full((4,), 0.9, device="cuda")
    outs = [torch.full((4,), -7, dtype=torch.int32, device="cuda") for _ in range(4)]
    st = torch.cuda.Stream()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=st):
        mk.sample(x, u, outs[0], top_k=k, top_p=p)
    torch.cuda.synchronize()
    gr.replay()
    mk.sample(x, u, outs[1], top_k=k, top_p=p)
    mk.sample(x, u, outs[2], top_k=k, top_p=p, stream=st)
    mk.sample(x, u, outs[3], top_k=k, top_p=p)
    torch.cuda.synchronize()
    assert all(torch.equal(o, outs[0]) for o in outs)


@pytest.mark.parametrize("vocab", [2045, 2048, 2049, 4093, 16384, 16387, 65536, 131069, 131070, 151936, 262144, 360448, 360446, 360449])
def test_sample_vocabularies_at_the_slices_edges(mk, vocab):
    sample_case(mk, noise(4, vocab, vocab), k=[0, 60, 0, 5], p=[1.0, 0.9, 0.9, 1.0], m=[0.0, 0.0, 0.0, 0.02])


def test_sample_large_k_and_flat_rows(mk):
    # beyond the candidates one block ranks: the exact cuts
    x = noise(6, 60000, 11, scale=0.02)
    sample_case(mk, x, k=[385, 5000, 59999, 400, 0, 384], p=[1.0, 0.5, 0.9, 0.99, 0.7, 1.0], t=[1.0, 2.0, 0.5, 1.0, 3e3, 1.0])
    x = noise(6, 60000, 12, scale=0.02, ties=True)
    sample_case(mk, x, k=[385, 5000, 59999, 400, 0, 384], p=[1.0, 0.5, 0.9, 0.99, 0.7, 1.0])


def test_sample_one_logit_far_above(mk):
    x = noise(5, 50000, 13)
    x[:, 49999] = 500.0
    sample_case(mk, x, k=[1, 50, 0, 0, 0], p=[1.0, 0.9, 0.9, 1.0, 1.0], m=[0.0, 0.0, 0.0, 0.5, 0.0])
    x[:, 7] = 500.0
    sample_case(mk, x, k=[1, 50, 0, 0, 0], p=[1.0, 0.9, 0.4, 1.0, 1.0], m=[0.0, 0.0, 0.0, 1.0, 0.0])


def test_sample_many_rows(mk):
    rng = np.random.default_rng(0)
    rows = 700
    k = [int(v) for v in rng.choice([0, 0, 5, 40], rows)]
    p = [float(v) for v in rng.choice([1.0, 0.6, 0.9], rows)]
    sample_case(mk, noise(rows, 3001, 14), k=k, p=p)
    # more rows than are put in order
    sample_case(mk, noise(3 * rows, 301, 15), k=3 * k, p=3 * p)


# ---- workspaces, shared pages, streams, both ways of the binding ------------------------

def test_one_workspace_for_calls_of_other_sizes(mk):
    g = gen(20)
    big = make_cache(mk, g, [9000, 10, 700], 2, 128, 16, torch.bfloat16)
    ws = mk.paged_attention_workspace(big, 8, 9000)
    for lens, nq, nkv, d in (([9000, 10, 700], 8, 2, 128), ([33], 4, 1, 64), ([5000, 5000], 16, 2, 64), ([9000, 10, 700], 8, 2, 128)):
        cache = big if len(lens) == 3 else make_cache(mk, g, lens, nkv, d, 16, torch.bfloat16)
        need = mk.paged_attention_workspace(cache, nq, max(lens))
        if need.numel() > ws.numel():
            ws = need
        q = torch.randn(len(lens), nq, d, generator=g, device="cuda").bfloat16()
        out = torch.empty_like(q)
        mk.paged_attention(cache, q, ints(lens), max(lens), out, ws)
        paged_check(cache, q, lens, out, d ** -0.5)
    torch.cuda.synchronize()
    assert int(ws[:1024].max()) == 0          # the counters are ready for the next call


def test_paged_sequences_that_share_pages(mk):
    # a common prefix of three pages, read by four sequences
    g = gen(21)
    cache = make_cache(mk, g, [48, 60, 70, 90], 2, 64, 16, torch.float16)
    cache.page_table[1:, :3] = cache.page_table[0, :3]
    q = torch.randn(4, 4, 64, generator=g, device="cuda").half()
    out = torch.empty_like(q)
    lens = [48, 60, 70, 90]
    mk.paged_attention(cache, q, ints(lens), 90, out)
    paged_check(cache, q, lens, out, 0.125)


@pytest.mark.parametrize("lens,max_len", [([0, 0, 0], 0), ([0] * 70, 16), ([1], 1)])
def test_paged_nothing_or_next_to_nothing(mk, lens, max_len):
    paged_case(mk, lens, 4, 2, 64, 16, torch.bfloat16, max_len=max_len)


def test_paged_in_place(mk):
    g = gen(25)
    lens = [3000, 17, 0, 900]
    cache = make_cache(mk, g, lens, 2, 128, 16, torch.bfloat16)
    q = torch.randn(4, 8, 128, generator=g, device="cuda").bfloat16()
    out = q.clone()
    mk.paged_attention(cache, out, ints(lens), 3000, out)
    paged_check(cache, q, lens, out, 128 ** -0.5)


def test_paged_max_len_beyond_the_table(mk):
    # one page of 16 a sequence: 50 tokens cannot be there
    with pytest.raises(mk.MkError) as e:
        paged_case(mk, [0] * 70, 4, 2, 64, 16, torch.bfloat16, max_len=50)
    assert e.value.status == mk.MK_ERR_INVALID


def test_prompt_many_sequences(mk):
    rng = np.random.default_rng(1)
    lens = [int(x) for x in rng.integers(0, 300, 200)]
    prompt_case(mk, lens, 4, 1, 64, torch.bfloat16, seed=1)
    prompt_case(mk, lens[:70], 3, 1, 128, torch.float16, seed=2)


def test_prompt_long_and_many_short(mk):
    # levels with one sequence, with few and with all of them, beyond 32 at a time
    rng = np.random.default_rng(2)
    lens = [int(x) for x in rng.integers(0, 140, 90)] + [2100] + [int(x) for x in rng.integers(0, 700, 40)] + [1, 0, 1290]
    prompt_case(mk, lens, 2, 1, 64, torch.bfloat16, seed=3)
    prompt_case(mk, lens, 3, 1, 64, torch.float16, seed=4)


def test_first_calls_of_a_process_are_captured():
    """Nothing an operator sets up at its first call is forbidden in a capture."""
    import subprocess
    import sys
    code = """
import torch
from persistent_decode_megakernel_02_b200 import mk
i = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
kc = torch.zeros(9, 2, 16, 64, device="cuda", dtype=torch.bfloat16)
cache = mk.PagedKV(kc, kc.clone(), i([[0, 1, 2, 3]]))
q, k, v = (torch.randn(60, h, 64, device="cuda").bfloat16() for h in (4, 2, 2))
cu, zero, lens, x, u = i([0, 60]), i([0]), i([60]), torch.randn(3, 999, device="cuda"), torch.rand(3, device="cuda")
qo, ko, out, o1, token = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(q[:1]), i([0, 0, 0])
ws = torch.zeros(1 << 24, dtype=torch.uint8, device="cuda")
def run():
    mk.kv_append(cache, q, k, v, cu, zero, 1e4, qo, ko)
    mk.prompt_attention(qo, ko, v, cu, 60, out)
    mk.paged_attention(cache, qo[59:], lens, 60, o1, ws)
    mk.sample(x, u, token)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    run()
g.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (qo, ko, out, o1, token)]
run()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, (qo, ko, out, o1, token)))
# the last prompt row and the one-token form see the same keys: both round their
# result once, the prompt form its weights too (bf16, half a step: 2^-9 each)
d = (out[59:].float() - o1.float()).abs().max()
assert d <= 3 * 2.0 ** -8 * v.float().abs().max(), d
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_offsets_beyond_32_bits(mk):
    """Rows and pages more than 2^32 elements from their buffers' starts."""
    n, nq, nkv, d, ps = 300, 4, 2, 64, 16
    g = gen(26)
    stride = 1 << 24
    buf = torch.empty(n * stride, device="cuda", dtype=torch.bfloat16)
    rows = lambda heads, at: buf.as_strided((n, heads, d), (stride, d, 1), at)
    q, k, v, out = rows(nq, 0), rows(nkv, 4096), rows(nkv, 8192), rows(nq, 12288)
    for x in (q, k, v):
        x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    per = 20
    pages = (1 << 32) // (nkv * ps * d) + per + 3
    kc = torch.empty(pages, nkv, ps, d, device="cuda", dtype=torch.bfloat16)
    table = torch.arange(pages - 1, pages - 1 - per, -1, device="cuda", dtype=torch.int32)[None].contiguous()
    table[0, 3] = 5
    cache = mk.PagedKV(kc, torch.empty_like(kc), table)
    status = ints([0])
    mk.kv_append(cache, q, k, v, ints([0, n]), ints([0]), 1e4, status=status)
    pos = torch.arange(n, device="cuda", dtype=torch.float64)
    e = torch.finfo(torch.bfloat16).eps
    ref, r = rotate64(q0, pos, 1e4)
    assert ((q.double() - ref).abs() <= e / 2 * ref.abs() + 2.0 ** -21 * r + 1e-7).all()
    ref, r = rotate64(k0, pos, 1e4)
    for p in range(n):
        got = kc[table[0, p // ps], :, p % ps]
        assert ((got.double() - ref[p]).abs() <= e / 2 * ref[p].abs() + 2.0 ** -21 * r[p] + 1e-7).all()
        assert torch.equal(cache.v[table[0, p // ps], :, p % ps], v0[p])
    mk.prompt_attention(q, k, v, ints([0, n]), n, out, status=status)
    prompt_check(q.contiguous(), k.contiguous(), v.contiguous(), [n], out.contiguous(), d ** -0.5)
    mk.paged_attention(cache, q[n - 1:], ints([n]), n, out[n - 1:], status=status)
    paged_check(cache, q[n - 1:].clone(), [n], out[n - 1:].clone(), d ** -0.5)
    assert int(status) == 0
    del buf, q, k, v, out, kc, cache
    torch.cuda.empty_cache()
    stride = 1 << 28
    x = torch.empty(18 * stride, device="cuda").as_strided((18, 40000), (stride, 1))
    x.copy_(noise(18, 40000, 27))
    sample_case(mk, x, k=[40] * 9 + [0] * 9, p=[0.9] * 18)
    del x
    torch.cuda.empty_cache()


def test_calls_at_once_on_two_streams(mk):
    # everything twice, on two streams at the same time, each with its own buffers
    g = gen(22)
    runs = []
    for i, st in enumerate([torch.cuda.Stream(), torch.cuda.Stream()]):
        lens = [1500 + 100 * i, 37, 0, 260]
        n, cu = sum(lens), cu_of(lens)
        cache = make_cache(mk, g, [m + 8 for m in lens], 2, 64, 16, torch.bfloat16)
        q, k, v = (torch.randn(n, h, 64, generator=g, device="cuda").bfloat16() for h in (8, 2, 2))
        x = noise(16, 32000, 30 + i)
        runs.append(dict(st=st, lens=lens, cu=ints(cu), start=ints([0] * 4), cache=cache, q=q, k=k, v=v, out=torch.empty_like(q),
                         q1=torch.randn(4, 8, 64, generator=g, device="cuda").bfloat16(), x=x, u=torch.rand(16, device="cuda"),
                         token=torch.zeros(16, dtype=torch.int32, device="cuda"), kk=ints([40] * 16), l=ints(lens),
                         ws=mk.paged_attention_workspace(cache, 8, 1500 + 100 * i)))
        with pytest.raises(mk.MkError):               # beyond the table
            mk.paged_attention_workspace(cache, 8, 1700)
    torch.cuda.synchronize()
    for _ in range(3):
        for r in runs:
            with torch.cuda.stream(r["st"]):
                r["qr"], r["kr"], r["o1"] = torch.empty_like(r["q"]), torch.empty_like(r["k"]), torch.empty_like(r["q1"])
                mk.kv_append(r["cache"], r["q"], r["k"], r["v"], r["cu"], r["start"], 1e4, r["qr"], r["kr"])
                mk.prompt_attention(r["qr"], r["kr"], r["v"], r["cu"], 1700, r["out"])
                mk.paged_attention(r["cache"], r["q1"], r["l"], max(r["lens"]), r["o1"], r["ws"])
                mk.sample(r["x"], r["u"], r["token"], top_k=r["kk"])
    torch.cuda.synchronize()
    for r in runs:
        prompt_check(r["qr"], r["kr"], r["v"], r["lens"], r["out"], 0.125)
        paged_check(r["cache"], r["q1"], r["lens"], r["o1"], 0.125)
        want = [sample_reference(a, 1.0, 40, 1.0, 0.0, b) for a, b in zip(r["x"].cpu().numpy(), r["u"].cpu().numpy())]
        assert r["token"].tolist() == want


def test_the_binding_s_two_ways_agree(mk, monkeypatch):
    """The compiled way and the ctypes way: the same bits."""
    g = gen(23)
    lens = [70, 0, 9]
    n = sum(lens)
    q, k, v = (torch.randn(n, h, 64, generator=g, device="cuda").half() for h in (4, 2, 2))
    cu, zero, x, u = ints(cu_of(lens)), ints([0, 0, 0]), noise(3, 999, 9), torch.rand(3, device="cuda")
    status = ints([0])

    def everything():
        kc = torch.zeros(9, 2, 16, 64, device="cuda", dtype=torch.float16)
        cache = mk.PagedKV(kc, kc.clone(), ints([[0, 1, 2, 3, 4], [8, 8, 8, 8, 8], [5, 8, 8, 8, 8]]))
        qo, ko, out, o1 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q), torch.empty_like(q[:3])
        token = torch.zeros(3, dtype=torch.int32, device="cuda")
        mk.kv_append(cache, q, k, v, cu, zero, 1e4, qo, ko, status=status)
        mk.prompt_attention(qo, ko, v, cu, 70, out, status=status)
        mk.paged_attention(cache, qo[:3], ints(lens), 70, o1, mk.paged_attention_workspace(cache, 4, 70), status=status)
        mk.sample(x, u, token, torch.full((3,), 0.7, device="cuda"), ints([5, 0, 9]), torch.full((3,), 0.9, device="cuda"),
                  torch.full((3,), 0.01, device="cuda"))
        kv = cache.k.clone()
        mk.kv_append(cache, None, k, v, cu, zero, 1e4)
        return [qo, ko, out, o1, token, kv, cache.k, cache.v]

    calls = []
    real = mk._fast

    class Counted:
        def __getattr__(self, name):
            def call(*a):
                st = getattr(real, name)(*a)
                calls.append((name, st))
                return st
            return call

    class Never:
        def __getattr__(self, name):
            return lambda *a: -1

    monkeypatch.setattr(mk, "_fast", Counted())
    one = everything()
    assert sorted(calls) == [("kv_append", 0), ("kv_append", 0), ("paged_attention", 0), ("prompt_attention", 0), ("sample", 0)]
    monkeypatch.setattr(mk, "_fast", Never())
    two = everything()
    assert int(status) == 0
    for a, b in zip(one, two):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_binding_refusals(mk):
    g = gen(24)
    cache = make_cache(mk, g, [40, 40], 2, 64, 16, torch.bfloat16)
    ok = lambda *shape, dtype=torch.bfloat16: torch.zeros(*shape, device="cuda", dtype=dtype)
    cu, st = ints([0, 1, 2]), ints([0, 0])
    k, q = ok(2, 2, 64), ok(2, 4, 64)
    ws = mk.paged_attention_workspace(cache, 4, 40)

    def append(**kw):
        a = dict(q=q.clone(), k=k.clone(), v=k.clone(), cu_tokens=cu, start_pos=st, rope_theta=1e4)
        a.update(kw)
        mk.kv_append(cache, **a)

    def paged(**kw):
        a = dict(q=q, kv_lens=st, max_len=40, out=q.clone(), workspace=ws)
        a.update(kw)
        mk.paged_attention(cache, **a)

    def prompt(**kw):
        a = dict(q=q, k=k, v=k, cu_seqlens=cu, max_len=2, out=q.clone())
        a.update(kw)
        mk.prompt_attention(**a)

    def sample(**kw):
        a = dict(logits=ok(2, 50, dtype=torch.float32), uniform=ok(2, dtype=torch.float32), token_out=ints([0, 0]))
        a.update(kw)
        mk.sample(**a)

    append(), paged(), prompt(), sample()
    bad = [(append, dict(k=k.half())), (append, dict(q=ok(2, 3, 64))), (append, dict(q=ok(3, 4, 64))), (append, dict(v=k.cpu())),
           (append, dict(k=ok(2, 64, 2).transpose(1, 2))), (append, dict(cu_tokens=ints([0, 1]))),
           (append, dict(cu_tokens=torch.zeros(3, dtype=torch.int64, device="cuda"))), (append, dict(rope_theta=0.5)),
           (append, dict(q=None, q_out=q)), (append, dict(status=ints([0, 0]))), (append, dict(q_out=ok(2, 4, 128)[..., ::2])),
           (append, dict(q=ok(2, 4 * 64 + 4)[:, 4:].unflatten(1, (4, 64)))),
           (paged, dict(out=q.half())), (paged, dict(kv_lens=ints([0]))), (paged, dict(max_len=1000)), (paged, dict(max_len=-1)),
           (paged, dict(max_len=(1 << 32) + 5)), (paged, dict(max_len=(1 << 32) + 5, workspace=None)), (prompt, dict(max_len=(1 << 32) + 5)),
           (prompt, dict(max_len=-1)), (prompt, dict(max_len=2.5)),
           (paged, dict(workspace=ws[:8])), (paged, dict(workspace=ws.cpu())), (paged, dict(scale=0.0)), (paged, dict(q=ok(2, 20, 64), out=ok(2, 20, 64))),
           (prompt, dict(k=ok(2, 3, 64), v=ok(2, 3, 64))), (prompt, dict(q=q.float())), (prompt, dict(out=ok(3, 4, 64))),
           (prompt, dict(cu_seqlens=ints([0])[:0])), (prompt, dict(scale=-1.0)), (prompt, dict(q=ok(2, 4, 32), k=ok(2, 2, 32), v=ok(2, 2, 32), out=ok(2, 4, 32))),
           (sample, dict(logits=ok(2, 50))), (sample, dict(logits=ok(2, 50, dtype=torch.float32).t())), (sample, dict(uniform=ok(3, dtype=torch.float32))),
           (sample, dict(top_k=ok(2, dtype=torch.float32))), (sample, dict(token_out=torch.zeros(2, dtype=torch.int64, device="cuda"))),
           (sample, dict(top_p=ok(4, dtype=torch.float32)[::2]))]
    for f, kw in bad:
        with pytest.raises(mk.MkError) as e:
            f(**kw)
        assert e.value.status == mk.MK_ERR_INVALID, kw
    torch.cuda.synchronize()


# ---- used together, and with the decode step ---------------------------------------------

def test_prompt_then_decode_over_pages(mk):
    """A prompt appended and attended in one call, then tokens appended and
    attended one at a time: every row as attention over the whole sequence."""
    nq, nkv, d, page, theta, dtype = 8, 2, 64, 16, 1e4, torch.bfloat16
    lens, steps = [37, 0, 130], 5
    g = gen(12)
    total = [n + steps for n in lens]
    rows = [[torch.randn(n, h, d, generator=g, device="cuda").to(dtype) for h in (nq, nkv, nkv)] for n in total]
    cache = make_cache(mk, g, total, nkv, d, page, dtype)
    cache.k.fill_(NAN)
    cache.v.fill_(NAN)
    q, k, v = (torch.cat([r[i][:n] for r, n in zip(rows, lens)]) for i in range(3))
    cu, zero = ints(cu_of(lens)), ints([0] * 3)
    kr, out = torch.empty_like(k), torch.empty_like(q)
    mk.kv_append(cache, q, k, v, cu, zero, theta, k_out=kr)
    mk.prompt_attention(q, kr, v, cu, max(lens), out)
    got = [[out[a:a + n]] for a, n in zip(cu_of(lens), lens)]
    one = ints([0, 1, 2, 3])
    for t in range(steps):
        q, k, v = (torch.stack([r[i][n + t] for r, n in zip(rows, lens)]) for i in range(3))
        mk.kv_append(cache, q, k, v, one, ints([n + t for n in lens]), theta)
        o = torch.empty_like(q)
        mk.paged_attention(cache, q, ints([n + t + 1 for n in lens]), max(total), o)
        for s in range(3):
            got[s].append(o[s:s + 1])
    e = torch.finfo(dtype).eps
    for s in range(3):
        pos = torch.arange(total[s], device="cuda")
        # the operators' inputs to attention are rotated rows rounded to bf16
        rq, rk = (rotate64(x, pos, theta)[0].to(dtype) for x in rows[s][:2])
        ref, mass = prompt_reference(rq, rk, rows[s][2], [total[s]], d ** -0.5)
        # a rotation that rounds the other way moves a score by up to e * |q||k| / sqrt(d) / sqrt(d) terms: ~ e * 8 / 8
        tol = e / 2 * ref.abs() + (e / 2 + 2.0 ** -11 + 2 * e) * mass
        assert ((torch.cat(got[s]).double() - ref).abs() <= tol).all(), s


@pytest.mark.parametrize("max_batch", [1, 3])
def test_operators_read_and_write_a_contexts_cache(mk, max_batch):
    """paged_attention over a context's own cache gives the step's attention;
    sampling its logits at temperature 0 gives its next token."""
    shape, S, n = wl.TINY, 48, 20
    w = wl.make_weights(shape, seed=5, device="cuda")
    kc, vc = wl.make_kv(shape, max_batch, S, device="cuda")
    ctx = mk.Context(w, kc, vc, S, max_batch)
    tok, pos, nxt = (torch.zeros(max_batch, dtype=torch.int32, device="cuda") for _ in range(3))
    logits = torch.zeros(max_batch, shape.vocab, device="cuda")
    sampled, u = torch.zeros_like(tok), torch.full((max_batch,), 0.5, device="cuda")
    zero, kk = torch.zeros(max_batch, device="cuda"), torch.full((max_batch,), 40, dtype=torch.int32, device="cuda")
    tok.copy_(ints([3, 5, 7][:max_batch]))
    for p in range(n):
        pos.fill_(p)
        ctx.decode_step(tok, pos, nxt, logits)
        mk.sample(logits, u, sampled, temperature=zero)
        assert ctx.sync() == 0 and torch.equal(sampled, nxt)
        mk.sample(logits, u, tok, top_k=kk)          # the next step's token, sampled
    last = shape.layers - 1
    cache = ctx.paged_kv(last)
    assert cache.k.data_ptr() == kc[last].data_ptr()
    if max_batch == 1:
        nq, d = shape.n_q_heads, shape.head_dim
        q = torch.from_numpy(ctx.read_buffer(mk.MK_BUF_Q, nq * d)).cuda().view(1, nq, d)
        want = torch.from_numpy(ctx.read_buffer(mk.MK_BUF_ATTN, nq * d)).cuda().view(1, nq, d).double()
        # rotate the query by appending into a scratch cache
        k = torch.zeros(3, shape.n_kv_heads, 16, d, device="cuda", dtype=torch.bfloat16)
        scratch = mk.PagedKV(k, k.clone(), ints([[0, 1, 2]]))
        row = torch.zeros(1, shape.n_kv_heads, d, device="cuda", dtype=torch.bfloat16)
        qb = q.bfloat16()
        mk.kv_append(scratch, qb, row, row, ints([0, 1]), ints([n - 1]), shape.rope_theta)
        out = torch.empty_like(qb)
        mk.paged_attention(cache, qb, ints([n]), n, out)
        # q rounded to bf16 twice and the output once; scores are O(1)
        assert (out.double() - want).abs().max() <= 4 * 2.0 ** -8 * want.abs().max()
    # and the other way: what kv_append writes, the step reads
    before = kc[last].clone()
    row = torch.ones(1, shape.n_kv_heads, shape.head_dim, device="cuda", dtype=torch.bfloat16)
    cu = [0] * max_batch + [1]
    mk.kv_append(cache, None, row, row, ints(cu), ints([n] * max_batch), shape.rope_theta)
    torch.cuda.synchronize()
    assert (vc[last][max_batch - 1, :, n] == 1).all()
    before[max_batch - 1, :, n] = kc[last][max_batch - 1, :, n]
    assert torch.equal(kc[last], before)
    ctx.close()


def test_decode_loop_in_one_graph(mk):
    """A serving loop's step -- append, attend, project, sample -- captured once and replayed
    while the positions grow and the sampled tokens feed the next step, as the same calls made
    one by one."""
    nq, nkv, d, page, vocab, seqs, steps = 4, 2, 64, 16, 500, 3, 20
    g = gen(31)
    table = ints([[s * 3 + i for i in range(3)] for s in range(seqs)])
    wq, wk, wv, wo = (torch.randn(vocab, h * d, generator=g, device="cuda").bfloat16() for h in (nq, nkv, nkv, nq))
    u = torch.rand(steps, seqs, generator=g, device="cuda")
    kk, pp = ints([30] * seqs), torch.full((seqs,), 0.95, device="cuda")
    one = ints([0, 1, 2, 3])

    def loop(graph):
        kc = torch.zeros(9, nkv, page, d, device="cuda", dtype=torch.bfloat16)
        cache = mk.PagedKV(kc, kc.clone(), table)
        token, pos, lens, un = ints([1, 2, 3]), ints([0, 5, 11]), ints([1, 6, 12]), torch.zeros(seqs, device="cuda")
        out = torch.empty(seqs, nq, d, device="cuda", dtype=torch.bfloat16)
        ws = mk.paged_attention_workspace(cache, nq, 3 * page)

        def step():
            t = token.long()
            q, k, v = wq[t].view(seqs, nq, d).clone(), wk[t].view(seqs, nkv, d), wv[t].view(seqs, nkv, d)
            mk.kv_append(cache, q, k, v, one, pos, 1e4)
            mk.paged_attention(cache, q, lens, 3 * page, out, ws)
            mk.sample(out.view(seqs, -1).float() @ wo.float().t(), un, token, None, kk, pp)
            pos.add_(1)
            lens.add_(1)

        if graph:
            st = torch.cuda.Stream()
            with torch.cuda.stream(st):
                for _ in range(2):
                    step()
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=st):
                step()
            kc.zero_(), cache.v.zero_()
            token.copy_(ints([1, 2, 3])), pos.copy_(ints([0, 5, 11])), lens.copy_(ints([1, 6, 12]))
        seen = []
        for i in range(steps):
            un.copy_(u[i])
            gr.replay() if graph else step()
            seen.append(token.clone())
        torch.cuda.synchronize()
        return torch.stack(seen), cache.k.clone(), cache.v.clone()

    for a, b in zip(loop(False), loop(True)):
        assert torch.equal(a, b)


# ---- single rows: their heads and elements are contiguous too ------------------------------

class FastNever:
    """Stands for the compiled way: nothing is taken."""

    def __getattr__(self, name):
        return lambda *a: -1


@pytest.mark.parametrize("fast", [True, False], ids=["compiled", "ctypes"])
@pytest.mark.parametrize("layout", ["interleaved", "transposed", "sliced", "expanded heads", "expanded elements"])
def test_single_rows_of_other_layouts_are_refused(mk, monkeypatch, fast, layout):
    if not fast:
        monkeypatch.setattr(mk, "_fast", FastNever())
    g = gen(40)
    cache = make_cache(mk, g, [40], 2, 64, 16, torch.bfloat16)
    ws = mk.paged_attention_workspace(cache, 4, 40)
    ok = lambda h: torch.zeros(1, h, 64, device="cuda", dtype=torch.bfloat16)
    z = lambda *shape: torch.zeros(*shape, device="cuda", dtype=torch.bfloat16)
    bad = {"interleaved": lambda h: z(1, h, 3, 64)[:, :, 1], "transposed": lambda h: z(1, 64, h).transpose(1, 2),
           "sliced": lambda h: z(1, h, 128)[..., :64], "expanded heads": lambda h: z(1, 1, 64).expand(1, h, 64),
           "expanded elements": lambda h: z(1, h, 1).expand(1, h, 64)}[layout]
    cu, start, lens = ints([0, 1]), ints([3]), ints([40])
    before = cache.k.clone(), cache.v.clone()
    calls = []
    for name, heads in (("q", 4), ("k", 2), ("v", 2), ("q_out", 4), ("k_out", 2)):
        a = dict(q=ok(4), k=ok(2), v=ok(2), q_out=ok(4), k_out=ok(2))
        a[name] = bad(heads)
        calls.append(lambda a=a: mk.kv_append(cache, a["q"], a["k"], a["v"], cu, start, 1e4, a["q_out"], a["k_out"]))
    for name in ("q", "out"):
        a = dict(q=ok(4), out=ok(4))
        a[name] = bad(4)
        calls.append(lambda a=a: mk.paged_attention(cache, a["q"], lens, 40, a["out"], ws))
    for name, heads in (("q", 4), ("k", 2), ("v", 2), ("out", 4)):
        a = dict(q=ok(4), k=ok(2), v=ok(2), out=ok(4))
        a[name] = bad(heads)
        calls.append(lambda a=a: mk.prompt_attention(a["q"], a["k"], a["v"], cu, 1, a["out"]))
    for call in calls:
        with pytest.raises(mk.MkError) as e:
            call()
        assert e.value.status == mk.MK_ERR_INVALID
    torch.cuda.synchronize()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))
    assert same(cache.k, before[0]) and same(cache.v, before[1])


@pytest.mark.parametrize("fast", [True, False], ids=["compiled", "ctypes"])
def test_single_rows_of_any_row_stride(mk, monkeypatch, fast):
    # one token of a fused buffer, whose row stride means nothing
    if not fast:
        monkeypatch.setattr(mk, "_fast", FastNever())
    g = gen(41)
    cache = make_cache(mk, g, [40], 2, 64, 16, torch.bfloat16)
    buf = torch.randn(1, 9, 64, generator=g, device="cuda").bfloat16()
    q, k, v = buf[:, :4].as_strided((1, 4, 64), (7, 64, 1)), buf[:, 4:6], buf[:, 6:8]
    q0, k0 = q.clone(), k.clone()
    out, ko, o = torch.empty_like(q0), torch.empty_like(k0), torch.empty_like(q0)
    mk.kv_append(cache, q, k, v, ints([0, 1]), ints([39]), 1e4, out, ko)
    for x, got in ((q0, out), (k0, ko)):
        ref, r = rotate64(x, torch.tensor([39], device="cuda"), 1e4)
        assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * r + 1e-7).all()
    mk.paged_attention(cache, q, ints([40]), 40, o, mk.paged_attention_workspace(cache, 4, 40))
    paged_check(cache, q0, [40], o, 0.125)
    mk.prompt_attention(q, k, v, ints([0, 1]), 1, o)
    prompt_check(q0, k0, v.contiguous(), [1], o, 0.125)


# ---- prompt attention: values that are not finite, broken offsets --------------------------

def seen_not_finite(v, lens, nq):
    """What a row's output must hold where it sees values that are not finite: NaN for a NaN or
    both infinities, else the infinity; 0 where all it sees is finite."""
    G, at = nq // v.shape[1], 0
    want = torch.zeros(v.shape[0], nq, v.shape[2], device="cuda")
    for n in lens:
        x = v[at:at + n]
        any_of = lambda m: m.long().cumsum(0) > 0
        nan, pos, neg = any_of(x.isnan()), any_of(x == INF), any_of(x == -INF)
        w = torch.where(pos, torch.full_like(want[at:at + n, :v.shape[1]], INF), torch.where(neg, -INF, 0.0))
        w = torch.where(nan | (pos & neg), NAN, w)
        want[at:at + n] = w.repeat_interleave(G, 1)
        at += n
    return want


def prompt_poison_case(mk, lens, nq, nkv, d, dtype, at, seed=0):
    """`at`: (row, KV head, column, value).  Rows that see one hold exactly what the formula gives
    (scores of N(0,1) inputs leave every weight far above zero); all others the clean run's bits."""
    q, k, v = prompt_inputs(lens, nq, nkv, d, dtype, seed)
    clean, out, status = torch.empty_like(q), torch.full_like(q, 7.0), ints([0])
    mk.prompt_attention(q, k, v, ints(cu_of(lens)), max(lens), clean)
    prompt_check(q, k, v, lens, clean, d ** -0.5)
    for row, h, col, x in at:
        v[row, h, col] = x
    mk.prompt_attention(q, k, v, ints(cu_of(lens)), max(lens), out, status=status)
    assert int(status) == 0
    want = seen_not_finite(v, lens, nq)
    assert torch.equal(out[want == 0], clean[want == 0])
    got = out.float()
    assert torch.equal(got[want.isinf()], want[want.isinf()]) and got[want.isnan()].isnan().all()


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("nq,nkv,d", [(2, 1, 64), (3, 1, 64), (6, 2, 128), (7, 1, 128), (4, 4, 64)])
def test_prompt_values_that_are_not_finite(mk, dtype, nq, nkv, d):
    # every column half and swizzle place, the last key of a tile, the first of the next, the very
    # last, NaN and infinities of both signs in one column and in different ones
    lens = [100, 300, 0, 257, 128]
    starts = cu_of(lens)
    at = [(starts[s] + r, c % nkv, c % d, x) for s, r, c, x in
          [(0, 0, 0, INF), (0, 40, 0, INF), (0, 41, 5, NAN), (0, 99, 63, -INF), (1, 40, 33, INF), (1, 60, 33, -INF), (1, 127, 7, INF),
           (1, 128, 8, -INF), (1, 255, 31, NAN), (1, 256, 32, INF), (1, 299, 64, NAN), (1, 290, 100, -INF), (3, 256, 127, INF),
           (3, 130, 95, -INF), (3, 200, 96, NAN), (4, 127, 17, INF), (4, 126, 17, INF)]]
    prompt_poison_case(mk, lens, nq, nkv, d, dtype, at, seed=nq)


@pytest.mark.parametrize("lens,nq,nkv,d", [([20] * 700, 2, 1, 64), ([150] * 500, 3, 1, 128), ([200, 10] * 200, 8, 2, 64)])
def test_prompt_values_that_are_not_finite_stay_with_their_item(mk, lens, nq, nkv, d):
    # a block takes several items one after another: what one left behind must not reach the next
    starts, rng = cu_of(lens), np.random.default_rng(len(lens))
    at = []
    for s in [*range(0, 150), *range(200, len(lens), 7)]:
        for _ in range(3):
            at.append((starts[s] + int(rng.integers(lens[s])), int(rng.integers(nkv)), int(rng.integers(d)),
                       [INF, -INF, NAN][int(rng.integers(3))]))
    prompt_poison_case(mk, lens, nq, nkv, d, torch.bfloat16, at, seed=1)


@pytest.mark.parametrize("cu", [[0, 10, 5, 20], [0, 10, 400, 20], [-4, 10, 15, 20], [0, 10, 15, 50], [3, 10, 15, 20]])
def test_prompt_rows_of_broken_offsets(mk, cu):
    # sequences that are whole are right, rows no such sequence claims stay
    n, top = 30, 16
    q, k, v = prompt_inputs([n], 2, 1, 64, torch.bfloat16)
    out = torch.full_like(q, 7.0)
    mk.prompt_attention(q, k, v, ints(cu), top, out)
    claims = [[] for _ in range(n)]
    for a, b in zip(cu, cu[1:]):
        if 0 <= a <= b <= n and b - a <= top:
            ref, mass = prompt_reference(q[a:b], k[a:b], v[a:b], [b - a], 0.125)
            tol = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -11) * mass + 1e-7
            for i, ok in enumerate((out[a:b].double() - ref).abs() <= tol):
                claims[a + i].append(ok)
    for i, c in enumerate(claims):        # of two claims each element has either's value
        assert torch.stack(c).any(0).all() if c else (out[i] == 7).all(), i


# ---- an error that an earlier call left behind ----------------------------------------------

def failed_create(mk):
    """A context whose head alone is larger than any device: mk_create returns MK_ERR_OOM."""
    from types import SimpleNamespace
    shape = wl.ModelShape(name="huge head", layers=1, hidden=2048, n_q_heads=4, n_kv_heads=4, head_dim=64, ffn=64, tied=False,
                          vocab=1 << 26, rope_theta=1e4, rms_eps=1e-5)
    x = torch.zeros(1 << 20, device="cuda", dtype=torch.bfloat16)
    w = SimpleNamespace(shape=shape, embed=x, lm_head=x, final_norm=x, **{n: [x] for n in (
        "attn_norm", "mlp_norm", "wq", "wk", "wv", "wo", "wg", "wu", "wd")})
    with pytest.raises(mk.MkError) as e:
        mk.Context(w, [x], [x], 16, 1)
    assert e.value.status == mk.MK_ERR_OOM


def test_a_failed_create_does_not_reach_the_next_calls(mk):
    # the failed allocation's error stays with the thread; a launch that went well must not be
    # reported (and made again: rows rotated in place would turn twice)
    g = gen(42)
    for form in range(5):
        cache = make_cache(mk, g, [40], 2, 64, 16, torch.bfloat16)
        q, k, v = (torch.randn(20, h, 64, generator=g, device="cuda").bfloat16() for h in (4, 2, 2))
        q0, k0 = q.clone(), k.clone()
        ws = mk.paged_attention_workspace(cache, 4, 40)
        out, o1, cu = torch.empty_like(q), torch.empty_like(q[:1]), ints([0, 20])
        x, token = noise(2, 999, 40), ints([-7, -7])
        xl, u = (noise(1, mk.MAX_VOCAB, 41) if form == 4 else None), torch.rand(2, device="cuda")
        torch.cuda.synchronize()
        failed_create(mk)
        if form == 0:
            mk.kv_append(cache, q, k, v, cu, ints([3]), 1e4, k_out=k)
            for a, got in ((q0, q), (k0, k)):
                ref, r = rotate64(a, torch.arange(3, 23, device="cuda"), 1e4)
                assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -21 * r + 1e-7).all()
        elif form == 1:
            mk.prompt_attention(q, k, v, cu, 20, out)
            prompt_check(q, k, v, [20], out, 0.125)
        elif form == 2:
            mk.paged_attention(cache, q[:1], ints([40]), 40, o1, ws)
            paged_check(cache, q[:1], [40], o1, 0.125)
        elif form == 3:
            mk.sample(x, u, token)
            assert (token >= 0).all()
        else:
            mk.sample(xl, u[:1], token[:1])
            assert token[0] >= 0
    # and through the library's own functions, which say MK_OK
    failed_create(mk)
    lens, o1 = ints([40]), torch.empty_like(q[:1])
    assert mk._lib.mk_paged_attention(cache._ref, lens.data_ptr(), 40, 4, q.data_ptr(), 256, 0.125, o1.data_ptr(), 256,
                                      ws.data_ptr(), ws.numel(), None, torch.cuda.current_stream().cuda_stream) == mk.MK_OK
    # a context that fits is made after one that did not
    failed_create(mk)
    w = wl.make_weights(wl.TINY, seed=5, device="cuda")
    kc, vc = wl.make_kv(wl.TINY, 2, 48, device="cuda")
    mk.Context(w, kc, vc, 48, 2).close()


# ---- many small weights beside a large one ---------------------------------------------------

def spiked_scores(n, d, dtype, heads_at, far):
    """Keys whose scores, in powers of two with scale = ln 2, are `far` at `heads_at` and 0 elsewhere;
    values 0 there and of both signs elsewhere, so that the small weights make the result."""
    k = torch.zeros(n, 1, d, device="cuda", dtype=dtype)
    k[heads_at, 0, 0] = far
    v = torch.ones(n, 1, d, device="cuda", dtype=dtype)
    v[:, 0, 1::2] = -0.75
    v[heads_at] = 0
    return k, v


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("far", [12.25, 16.75, 19.625, 20.375, 22.625, 24.625, 25.5, 27.0])
@pytest.mark.parametrize("d", [64, 128])
def test_paged_small_weights_are_kept(mk, dtype, far, d):
    # 400 sequences over the same pages: a block has whole sequences, its warps every 8th (64 dims)
    # or 6th step, and one large key each.  The tolerance is paged_check's, whose |v| has no share
    # of the large keys.
    n, page, seqs = 8192, 64, 400
    step, warps = (32, 8) if d == 64 else (16, 6)
    k, v = spiked_scores(n, d, dtype, [step * w + 3 for w in range(warps)], far)
    pages = lambda x: x.view(n // page, page, 1, d).transpose(1, 2).contiguous()
    cache = mk.PagedKV(pages(k), pages(v), torch.arange(n // page, device="cuda", dtype=torch.int32).repeat(seqs, 1))
    q = torch.zeros(seqs, 2, d, device="cuda", dtype=dtype)
    q[:, :, 0] = 1
    out = torch.empty_like(q)
    mk.paged_attention(cache, q, ints([n] * seqs), n, out, scale=math.log(2))
    ref, mass = paged_reference(cache, q[:1], [n], math.log(2))
    e = torch.finfo(dtype).eps
    assert ((out.double() - ref).abs() <= e / 2 * ref.abs() + 2.0 ** -11 * mass + 1e-7).all(), (out[0, 0, :2], ref[0, 0, :2])
    # and the large keys spread so that a warp meets one after many small ones
    k, v = spiked_scores(n, d, dtype, [n - 1 - step * w for w in range(warps)], far)
    cache.k.copy_(pages(k)), cache.v.copy_(pages(v))
    mk.paged_attention(cache, q, ints([n] * seqs), n, out, scale=math.log(2))
    assert ((out.double() - ref).abs() <= e / 2 * ref.abs() + 2.0 ** -11 * mass + 1e-7).all(), (out[0, 0, :2], ref[0, 0, :2])


# ---- paged attention: visible values that are not finite -------------------------------------

@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("nq,nkv,d,page", [(8, 2, 64, 16), (8, 1, 128, 7), (3, 3, 64, 64), (4, 2, 128, 16)])
def test_paged_values_that_are_not_finite(mk, dtype, nq, nkv, d, page):
    # a column that sees an infinity holds it, one with a NaN or both signs NaN, every other the
    # clean run's bits (the scores leave every weight far above zero)
    lens = [1, 700, 40, 5000, 0, 33, 64]
    g = gen(50 + d)
    cache = make_cache(mk, g, lens, nkv, d, page, dtype)
    q = torch.randn(len(lens), nq, d, generator=g, device="cuda").to(dtype)
    clean, out = torch.empty_like(q), torch.full_like(q, 7.0)
    mk.paged_attention(cache, q, ints(lens), max(lens), clean)
    paged_check(cache, q, lens, clean, d ** -0.5)
    want = torch.zeros(len(lens), nkv, d, device="cuda")
    table = cache.page_table.tolist()
    at = [(0, 0, 0, INF), (1, 0, 3, -INF), (1, 699, 4, INF), (1, 350, 5, NAN), (1, 17, 6, INF), (1, 500, 6, -INF), (1, 699, 63, -INF),
          (2, 39, 31, INF), (3, 0, 1, INF), (3, 4999, 2, -INF), (3, 2500, 62, INF), (3, 2501, 62, INF), (3, 16, d - 1, NAN), (5, 32, d // 2, -INF),
          (6, 63, 8, INF)]
    for s, p, c, x in at:
        h = c % nkv
        cache.v[table[s][p // page], h, p % page, c] = x
        w = want[s, h, c]
        want[s, h, c] = x if w == 0 or w == x else NAN
    mk.paged_attention(cache, q, ints(lens), max(lens), out)
    want = want.repeat_interleave(nq // nkv, 1)
    got = out.float()
    assert torch.equal(got[want.isinf()], want[want.isinf()]) and got[want.isnan()].isnan().all()
    assert torch.equal(out[want == 0], clean[want == 0])


@pytest.mark.parametrize("far", [35.0, 42.0, 60.0])
def test_paged_infinite_values_under_sharp_scores(mk, far):
    # weights of one and of next to nothing (2^-far) times an infinity, and finite columns beside
    # them as without it
    n, d, page = 600, 64, 16
    for dtype in DT.values():
        k, v = spiked_scores(n, d, dtype, [5], far)
        pages = lambda x: torch.cat([x, x[:608 - n]]).view(608 // page, page, 1, d).transpose(1, 2).contiguous()
        cache = mk.PagedKV(pages(k), pages(v), torch.arange(608 // page, device="cuda", dtype=torch.int32)[None].contiguous())
        q = torch.zeros(1, 2, d, device="cuda", dtype=dtype)
        q[:, :, 0] = 1
        clean, out = torch.empty_like(q), torch.empty_like(q)
        mk.paged_attention(cache, q, ints([n]), n, clean, scale=math.log(2))
        cache.v[0, 0, 5, 3], cache.v[0, 0, 6, 4], cache.v[0, 0, 5, 6], cache.v[20, 0, 1, 6] = INF, -INF, INF, -INF
        mk.paged_attention(cache, q, ints([n]), n, out, scale=math.log(2))
        assert (out[0, :, 3] == INF).all() and (out[0, :, 4] == -INF).all() and out[0, :, 6].isnan().all()
        rest = [i for i in range(d) if i not in (3, 4, 6)]
        assert torch.equal(out[..., rest], clean[..., rest])


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("far", [12.25, 16.75, 19.625, 20.375, 22.625, 24.625, 25.5])
@pytest.mark.parametrize("d", [64, 128])
def test_prompt_small_weights_are_kept(mk, dtype, far, d):
    # one large key at the start of a long prompt (and, rows apart, in its middle) and small weights
    # for all others, which make the result
    n = 3000
    for at in ([3], [1500, 1700]):
        k, v = spiked_scores(n, d, dtype, at, far)
        q = torch.zeros(n, 2, d, device="cuda", dtype=dtype)
        q[:, :, 0] = 1
        out = torch.empty_like(q)
        mk.prompt_attention(q, k, v, ints([0, n]), n, out, scale=math.log(2))
        prompt_check(q, k, v, [n], out, math.log(2))


# exponents whose power of two lies near the middle of two 16-bit values
DOWN = {"bf16": [0.9609375, 0.8046875, 0.578125], "fp16": [0.9921875, 0.9453125, 0.8046875]}


@pytest.mark.parametrize("dtype,down", [(torch.bfloat16, x) for x in DOWN["bf16"]] + [(torch.float16, x) for x in DOWN["fp16"]], ids=str)
@pytest.mark.parametrize("d", [64, 128])
def test_paged_weights_keep_their_remainder(mk, dtype, down, d):
    # Every 16th key scores 0 with value 0, all others -down (powers of two), so that each weight is
    # off by the same share when it is rounded to 16 bits.  Beyond the output's rounding: the two
    # parts hold a weight to 2^-16, ex2 to 2^-22, a score's 32-bit scaling to 2^-23, and 512 products
    # added in 32 bits lose at most 512 * 2^-24 = 2^-15: below 2^-14 in all.
    n, page = 4096, 64
    g = gen(60)
    k = torch.zeros(n, 1, d, device="cuda", dtype=dtype)
    k[:, 0, 0] = -down
    k[::16] = 0
    v = (0.5 + torch.rand(1, 1, d, generator=g, device="cuda")).to(dtype).repeat(n, 1, 1)
    v[::16] = 0
    pages = lambda x: x.view(n // page, page, 1, d).transpose(1, 2).contiguous()
    cache = mk.PagedKV(pages(k), pages(v), torch.arange(n // page, device="cuda", dtype=torch.int32)[None].contiguous())
    q = torch.zeros(1, 3, d, device="cuda", dtype=dtype)
    q[:, :, 0] = 1
    out = torch.empty_like(q)
    mk.paged_attention(cache, q, ints([n]), n, out, scale=math.log(2))
    ref, mass = paged_reference(cache, q, [n], math.log(2))
    fine = lambda x: ((x.double() - ref).abs() <= torch.finfo(dtype).eps / 2 * ref.abs() + 2.0 ** -14 * mass).all()
    assert fine(out)
    w = 2.0 ** -down         # and the check sees a weight that is rounded once
    assert fine(ref.to(dtype)) and not fine((ref * (float(torch.tensor(w).to(dtype)) / w)).to(dtype))


@pytest.mark.parametrize("dtype", DT.values(), ids=DT.keys())
@pytest.mark.parametrize("d", [64, 128])
def test_scores_of_minus_infinity_only(mk, dtype, d):
    # zeros where nothing but such keys is seen, the formula where one finite score joins them
    g = gen(61)
    n, page = 200, 16
    q = torch.ones(n, 2, d, device="cuda", dtype=dtype)
    k, v = (torch.randn(n, 1, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    k[:150, :, 3] = -INF
    out, status = torch.full_like(q, NAN), ints([0])
    mk.prompt_attention(q, k, v, ints([0, n]), n, out, status=status)
    assert (out[:150] == 0).all()
    prompt_check(q[150:], k[150:], v[150:], [n - 150], out[150:], d ** -0.5)
    pad = lambda x: torch.cat([x, x[:8]]).view(13, page, 1, d).transpose(1, 2).contiguous()
    cache = mk.PagedKV(pad(k), pad(v), torch.arange(13, device="cuda", dtype=torch.int32).repeat(4, 1))
    lens = [1, 150, 151, 200]
    o = torch.full_like(q[:4], NAN)
    mk.paged_attention(cache, q[:4].contiguous(), ints(lens), n, o, status=status)
    assert (o[:2] == 0).all() and int(status) == 0
    paged_check(cache, q[:4], lens, o, d ** -0.5, sel=[2, 3])
