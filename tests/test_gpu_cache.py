"""The cache operators on the GPU against the plain implementation in 64 bits of tests/_cache.py."""
import math

import numpy as np
import pytest
import torch

from _cache import TYPES, Step, append, attention, check_append, check_attention, cuda, off_by, ref_append, ref_attention

pytestmark = pytest.mark.gpu

PAIRS = (("bf16", "bf16"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "e4m3"))
LENGTHS = [0, 1, 15, 16, 63, 64, 65, 200, 127, 128, 700, 31]
NEW = [1, 2, 3, 6, 1, 4, 8, 5, 2, 1, 6, 3]


def freqs(m, theta=10000.0):
    return (theta ** (-torch.arange(m, dtype=torch.float64) / m)).float()


# ---------------------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("dim,rotary", ((64, 64), (128, 64), (256, 256), (16, 16), (80, 32), (96, 96), (128, 0)))
@pytest.mark.parametrize("interleaved", (False, True))
def test_append(dtype, cache, dim, rotary, interleaved):
    s = Step(dim + rotary, LENGTHS, NEW, hq=6, hk=3, dim=dim, dtype=dtype, cache=cache, page=16, layout="heads")
    check_append(s, inv_freq=freqs(rotary // 2) if rotary else None, interleaved=interleaved)


@pytest.mark.parametrize("page,layout", ((1, "tokens"), (5, "heads"), (48, "both"), (64, "both"), (128, "tokens"), (1000, "heads")))
def test_append_pages_and_layouts(page, layout):
    s = Step(page, LENGTHS, NEW, hq=8, hk=2, dim=128, page=page, layout=layout, spare=2)
    check_append(s, inv_freq=freqs(64, 500000.0))


def test_append_far_positions_and_axes():
    """Angles of positions up to 2^31: they are known to 2^-16 radians there and to 2^-27 at 2^20."""
    s = Step(3, [1000, 0, 77], [4, 9, 3], dim=128, hq=4, hk=1)
    g = torch.Generator().manual_seed(4)
    positions = torch.randint(0, 2**31 - 1, (3, s.rows), generator=g).int()
    positions[0, :4] = torch.tensor([0, 1, 2**20, 2**31 - 1], dtype=torch.int32)
    positions[1, :2] = torch.tensor([-5, -2**31], dtype=torch.int32)
    for axes in ([0] * 16 + [1] * 24 + [2] * 24, [m % 3 for m in range(64)], [2] * 64, None):
        check_append(s, inv_freq=freqs(64, 500000.0), positions=positions, axes=axes)
    check_append(s, inv_freq=torch.tensor([-1.5, 100.0, 7.0, 0.0, 1e-30, 3.0, -0.001, 1e6]), positions=positions[:1])
    check_append(s, inv_freq=freqs(8), positions=positions[2])


@pytest.mark.parametrize("rows,hq,hk", ((1, 32, 8), (1, 0, 1), (3, 1, 1), (700, 5, 1), (2500, 8, 2)))
def test_append_one_row_a_request(rows, hq, hk):
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(rows, [i * 7 % 40 for i in range(rows)], [1] * rows, hq=max(hq, 1), hk=hk, dim=64)
    k, v = s.device_caches()
    q = sv.cache_append(cuda(s.k), cuda(s.v), k, v, cuda(s.table), cuda(s.lengths), q=cuda(s.q) if hq else None, inv_freq=cuda(freqs(32)))
    want, err = ref_append(s, freqs(32))
    assert (q is None) == (hq == 0)
    for name, g, w, e in (("q", q, want[0], err[0]), ("k", k, want[1], err[1]), ("v", v, want[2], err[2])):
        if g is not None:
            off_by(g, w, e, name)


def test_append_leaves_out_what_takes_no_part():
    """Requests of negative length, bad pages, rows behind the last request's, places behind the table: nothing is written."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(9, [5, -1, 20, -2**31, 3, 60], [2, 3, 4, 1, 6, 6], dim=64, page=16)
    s.table[2, 1] = s.pool          # (places 16 to 23 of request 2)
    s.table[4, 0] = -7
    s.table = s.table[:, :4]        # (places from 64 on)
    s.width = 4
    check_append(s, inv_freq=freqs(32))
    more = 5
    k, v = s.device_caches()
    wide = lambda t: torch.cat((t, torch.full((more, *t.shape[1:]), 3.0, dtype=t.dtype))).cuda()  # noqa: E731
    out = torch.full((s.rows + more, s.hq, s.dim), 9.0, dtype=s.dtype, device="cuda")
    got = sv.cache_append(wide(s.k), wide(s.v), k, v, cuda(s.table), cuda(s.lengths), q=wide(s.q), inv_freq=cuda(freqs(32)), cu_num_draft=cuda(s.cu), out=out)
    want, err = ref_append(s, freqs(32))
    assert got is out and bool((out[s.rows:] == 9).all())
    off_by(out[:s.rows], want[0], err[0], "q")
    off_by(k, want[1], err[1], "k")
    for r, i, _ in s.rows_of():
        if int(s.lengths[i]) < 0:
            assert bool((out[r] == 9).all())


def test_append_views_of_a_projection_and_in_place():
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(11, [30, 2, 9], [3, 1, 7], hq=6, hk=2, dim=64, page=5)
    qkv = torch.cat((s.q.flatten(1), s.k.flatten(1), s.v.flatten(1)), 1).cuda()
    q, k, v = (x.view(s.rows, -1, 64) for x in qkv.split((6 * 64, 2 * 64, 2 * 64), 1))
    kc, vc = s.device_caches()
    got = sv.cache_append(k, v, kc, vc, cuda(s.table), cuda(s.lengths), q=q, inv_freq=cuda(freqs(32)), cu_num_draft=cuda(s.cu), out=q)
    assert got is q
    want, err = ref_append(s, freqs(32))
    for name, g, w, e in zip("qkv", (q, kc, vc), want, err):
        off_by(g, w, e, name)
    torch.testing.assert_close(qkv[:, 6 * 64:], torch.cat((s.k.flatten(1), s.v.flatten(1)), 1).cuda(), rtol=0, atol=0)


def test_append_8_bits_saturate_and_keep_nan():
    s = Step(12, [0], [4], hq=1, hk=1, dim=16, cache="e4m3")
    s.k_scale, s.v_scale = torch.tensor([0.001]), torch.tensor([2.0])
    s.v[0, 0, 0], s.v[1, 0, 0], s.v[2, 0, 0], s.v[3, 0, 0] = float("inf"), -float("inf"), float("nan"), 1e-30
    _, k, v = append(s)
    k, v = k.cpu().float(), v.cpu().float()
    got = [float(v[s.slot(0, x)][0, 0]) for x in range(4)]
    assert got[0] == 448 and got[1] == -448 and np.isnan(got[2]) and got[3] == 0
    assert float(k[s.slot(0, 0)].abs().max()) == 448
    # and without scales
    s.k_scale = s.v_scale = None
    check_append(Step(13, [3], [5], dim=32, cache="e4m3", hq=2, hk=2), inv_freq=freqs(16))


# ------------------------------------------------------------------------------- attention

@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("dim", (64, 128, 256))
@pytest.mark.parametrize("hq,hk", ((8, 2), (7, 1), (3, 3), (16, 1)))
def test_attention(dtype, cache, dim, hq, hk):
    check_attention(Step(dim + hq, LENGTHS, NEW, hq=hq, hk=hk, dim=dim, dtype=dtype, cache=cache, page=16, layout="heads", share=1.5))


@pytest.mark.parametrize("page,layout", ((1, "tokens"), (5, "heads"), (20, "both"), (64, "both"), (128, "tokens"), (1000, "heads")))
@pytest.mark.parametrize("dtype,cache", (("bf16", "bf16"), ("bf16", "e4m3")))
def test_attention_pages_and_layouts(page, layout, dtype, cache):
    check_attention(Step(page, LENGTHS, NEW, hq=8, hk=2, dim=128, dtype=dtype, cache=cache, page=page, layout=layout, spare=3))


@pytest.mark.parametrize("page", (15, 17, 18, 42, 72, 96, 100, 128, 129, 200))
@pytest.mark.parametrize("dim", (64, 128, 256))
def test_attention_8_bits_of_odd_pages(page, dim):
    """Pages that tensor maps bring to shared memory, and pages too small, beside 128 bytes, or a bad fit for a tile."""
    check_attention(Step(page + dim, LENGTHS, NEW, hq=6, hk=2, dim=dim, cache="e4m3", page=page, layout="heads", spare=1))


@pytest.mark.parametrize("window", (1, 2, 5, 16, 64, 100, 300, 10**9))
@pytest.mark.parametrize("dim,cache", ((64, "bf16"), (128, "e4m3")))
def test_attention_window(window, dim, cache):
    check_attention(Step(window % 97, LENGTHS, NEW, hq=8, hk=2, dim=dim, cache=cache, page=20), window=window)


@pytest.mark.parametrize("hq,hk,new", ((8, 1, [40, 3]), (4, 2, [100, 64]), (64, 2, [9, 8]), (1, 1, [1, 200]), (40, 1, [7, 1])))
@pytest.mark.parametrize("window", (0, 30))
def test_attention_of_many_rows(hq, hk, new, window):
    """More query rows to a key head than a tile holds: chunks of a prompt, wide groups."""
    check_attention(Step(hq, [50, 300], new, hq=hq, hk=hk, dim=64), window=window)
    check_attention(Step(hq, [0, 7], new, hq=hq, hk=hk, dim=256, dtype="f16", cache="f16"), window=window)


@pytest.mark.parametrize("lengths", ([5000], [3000, 2, 2500], [0], [1], [63], [64], [2047, 2048, 2049]))
@pytest.mark.parametrize("new", (1, 4))
def test_attention_split_over_the_length(lengths, new):
    for dim, dtype, cache in ((128, "bf16", "bf16"), (64, "f16", "f16"), (256, "bf16", "e4m3")):
        check_attention(Step(len(lengths), lengths, [new] * len(lengths), hq=4, hk=1, dim=dim, dtype=dtype, cache=cache, page=64), dim)


@pytest.mark.parametrize("n", (1, 33, 600, 2100))
def test_attention_many_requests(n):
    s = Step(n, [i * 37 % 90 for i in range(n)], [1 + i % 3 for i in range(n)], hq=4, hk=1, dim=64)
    check_attention(s)


@pytest.mark.parametrize("dim,hq,hk", ((256, 8, 1), (256, 16, 1), (128, 8, 1), (128, 12, 1), (128, 16, 1), (64, 24, 1)))
@pytest.mark.parametrize("cache,page", (("bf16", 32), ("e4m3", 32), ("bf16", 8), ("e4m3", 8)))
def test_attention_long_runs_of_tiles(dim, hq, hk, cache, page):
    """Hundreds of tiles of many requests for every CTA: rings of copies that go round many times."""
    import speculative_decoding_verification_rejection_gb300 as sv

    n, width = 96, 3200 // page
    g = torch.Generator(device="cuda").manual_seed(dim + hq)
    pages = torch.randn(300, page, hk, dim, generator=g, device="cuda")
    k, v = pages.to(TYPES[cache]), pages.flip(0).to(TYPES[cache])
    table = torch.randint(0, 300, (n, width), generator=g, device="cuda").int()
    lengths = torch.randint(0, 3100, (n,), generator=g, device="cuda").int()
    lengths[::7] = torch.arange(14, device="cuda").int()
    new = 4
    cu = torch.arange(n + 1, device="cuda").int() * (new - 1)
    q = torch.randn(n * new, hq, dim, generator=g, device="cuda").bfloat16()
    for _ in range(3):
        out, lse = sv.cache_attention(q, k, v, table, lengths, cu_num_draft=cu, lse=True)
    kk, vv = (c[table.long()].float().view(n, -1, dim).double() for c in (k, v))
    score = torch.einsum("nrhd,ntd->nrht", q.view(n, new, hq, dim).double(), kk) * dim ** -0.5
    seen = torch.arange(width * page, device="cuda") <= lengths[:, None, None].long() + torch.arange(new, device="cuda")[:, None]
    score.masked_fill_(~seen[:, :, None], -float("inf"))
    want = torch.einsum("nrht,ntd->nrhd", torch.softmax(score, -1), vv)
    # the largest value's weights off by one rounding of 16 bits (2^-8), the output's likewise
    assert float((out.view(n, new, hq, dim).double() - want).abs().max()) <= float(vv.abs().max()) * 2.0**-7
    assert float((lse.view(n, new, hq).double() - torch.logsumexp(score, -1)).abs().max()) <= 1e-4   # (scores up to 10, 2^-22 each of 128 products)


@pytest.mark.parametrize("scale", (0.0, -0.3, 1e-20, 2.0))
def test_attention_scale(scale):
    check_attention(Step(5, [100, 3], [2, 5], dim=128), scale=scale)
    check_attention(Step(6, [100, 3], [2, 5], dim=64, cache="e4m3"), scale=scale)


def test_attention_without_a_key():
    """Requests of negative length, pages that are not there: rows that see nothing, and tiles in part."""
    s = Step(21, [5, -1, 120, -2**31, 3, 60], [2, 3, 4, 1, 6, 6], dim=64, page=16)
    s.table[2, 1:4] = torch.tensor([s.pool, -1, 2**31 - 1])
    s.table[4, 0] = -7
    s.table = s.table[:, :7]
    s.width = 7
    check_attention(s)
    check_attention(s, window=9)
    none = Step(22, [4], [3], dim=128)
    none.table = none.table[:, :0].contiguous()
    none.width = 0
    check_attention(none)


@pytest.mark.parametrize("dtype,cache", PAIRS)
@pytest.mark.parametrize("bad", (float("nan"), float("inf"), -float("inf")))
def test_what_is_not_seen_does_not_matter(dtype, cache, bad):
    """All of the pool but the seen slots, and for the first rows the later ones' keys and values, hold NaN or infinities."""
    if cache == "e4m3":
        bad = float("nan")
    for window in (0, 3):
        s = Step(31, [0, 40, 65, 130], [6, 5, 8, 2], dim=64, hq=6, hk=2, dtype=dtype, cache=cache, page=16)
        clean = [c.clone() for c in (s.k_cache, s.v_cache)]
        for c in (s.k_cache, s.v_cache):
            c.view(torch.uint8).copy_(torch.full_like(c.float(), bad).to(c.dtype).view(torch.uint8))
        for i in range(s.n):
            for x in range(int(s.lengths[i]) + 1):  # what the first row sees
                if window and x <= int(s.lengths[i]) - window:
                    continue
                for c, was in zip((s.k_cache, s.v_cache), clean):
                    c[s.slot(i, x)] = was[s.slot(i, x)]
        out, lse = attention(s, window=window)
        (want, want_lse), (oe, le) = ref_attention(s, window=window)
        for i in range(s.n):
            r = s.first[i]
            off_by(out[r], want[r], oe[r], f"request {i}")
            off_by(lse[r], want_lse[r], le[r], f"request {i} lse")
        last = [s.first[i] + s.new[i] - 1 for i in range(s.n)]
        assert bool(torch.isnan(out[last]).all())   # (and a row that sees them shows it)


def test_nan_and_infinite_scores():
    """A key whose score is -inf does not count, a row with only such keys is empty; NaN and +inf make NaN."""
    s = Step(41, [20, 20, 20, 20], [1] * 4, dim=64, hq=2, hk=1, page=32)
    s.q.fill_(1.0)
    for x in range(21):
        s.k_cache[s.slot(0, x)] = -float("inf")
        if x != 7:
            s.k_cache[s.slot(1, x)] = -float("inf")
    s.k_cache[s.slot(2, 3)] = float("nan")
    s.k_cache[s.slot(3, 3)] = float("inf")
    out, lse = (t.cpu().float() for t in attention(s))
    assert bool((out[0] == 0).all()) and bool((lse[0] == -float("inf")).all())
    torch.testing.assert_close(out[1], s.v_cache[s.slot(1, 7)].float().expand(2, 64), rtol=0, atol=0)
    assert bool(torch.isnan(out[2:]).all())


def test_far_off_scores_and_values():
    """Scores in the thousands, a cancelling pair, tiny queries beside large ones (8-bit cache)."""
    s = Step(42, [500, 90], [2, 3], dim=128, hq=4, hk=2, share=300.0)
    check_attention(s)
    s = Step(43, [500, 90], [2, 3], dim=128, hq=4, hk=2, cache="e4m3")
    s.q *= torch.logspace(-12, 6, s.dim).bfloat16()
    check_attention(s)
    s.q[0] = 0
    s.q[1] *= 2.0**-100
    check_attention(s)
    s = Step(44, [500, 90], [2, 3], dim=64, dtype="f16", cache="f16")
    s.v_cache *= 2000
    check_attention(s)


def test_many_keys_of_small_weight_count():
    """One key of weight 1 and 60000 of weight 2^-20 to 2^-30: their sum is not lost in 16 bits."""
    for dtype, cache in (("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3")):
        s = Step(45, [60000], [1], dim=64, hq=1, hk=1, dtype=dtype, cache=cache, page=128)
        s.k_scale = s.v_scale = None
        k, v = torch.zeros(s.k_cache.shape), torch.ones(s.v_cache.shape)
        k[s.slot(0, 30000)][0, 0], v[s.slot(0, 30000)][0] = 18.0, -1.0
        s.k_cache, s.v_cache = k.to(s.kind), v.to(s.kind)
        s.q.zero_()
        s.q[0, 0, 0] = 1.0
        check_attention(s, scale=1.0)


def test_attention_strides_and_rows_behind():
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(51, LENGTHS, NEW, hq=8, hk=2, dim=64)
    more = 7
    wide = torch.full((s.rows + more, 3, 8, 80), 7.0, dtype=s.dtype, device="cuda")
    wide[:s.rows, 1, :, 8:72] = s.q.cuda()
    out = torch.full((8, s.rows + more, 72), 5.0, dtype=s.dtype, device="cuda")
    k, v = s.device_caches()
    got = sv.cache_attention(wide[:, 1, :, 8:72], k, v, cuda(s.table), cuda(s.lengths), cu_num_draft=cuda(s.cu), out=[out.transpose(0, 1)[..., :64]])
    want, err = ref_attention(s)
    off_by(got[0][:s.rows], want[0], err[0], "out")
    assert bool((out[:, s.rows:] == 5).all()) and bool((out[:, :, 64:] == 5).all())
    # a page table that is a view of a wider one
    table = torch.full((s.n, 2 * s.width + 1), -3, dtype=torch.int32, device="cuda")
    table[:, 1:1 + s.width] = s.table.cuda()
    again, = sv.cache_attention(cuda(s.q), k, v, table[:, 1:1 + s.width], cuda(s.lengths), cu_num_draft=cuda(s.cu))
    off_by(again, want[0], err[0], "a view of a page table")   # (other sizes may be split otherwise)


def test_one_row_a_request_without_prefix_sums():
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(52, LENGTHS, [1] * len(LENGTHS), hq=4, hk=4, dim=128)
    k, v = s.device_caches()
    got = sv.cache_attention(cuda(s.q), k, v, cuda(s.table), cuda(s.lengths), lse=True)
    with_sums = attention(s, (k, v))
    want, err = ref_attention(s)
    for a, b, w, e in zip(got, with_sums, want, err):
        off_by(a, w, e, "one row a request")
        torch.testing.assert_close(a, b, rtol=0, atol=0)


@pytest.mark.parametrize("cu", ([0, 1, 0, 5], [0, -3, 2, 5], [0, 2, 2**31 - 1, 5], [-2**31, 0, 1, 2], [0, 100, 100, 100], [7, 7, 7, 7]))
def test_inconsistent_prefix_sums_stay_inside(cu):
    """Rows of requests that are not within the batch are left out; the consistent ones are right."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(53, [10, 20, 30], [2, 1, 5], dim=64)
    k, v = s.device_caches()
    out = torch.full((s.rows, s.hq, s.dim), 5.0, dtype=s.dtype, device="cuda")
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    sv.cache_attention(cuda(s.q), k, v, cuda(s.table), cuda(s.lengths), cu_num_draft=bad, out=[out])
    sv.cache_append(cuda(s.k), cuda(s.v), k, v, cuda(s.table), cuda(s.lengths), cu_num_draft=bad)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out).all())


def test_results_repeat_bit_for_bit():
    s = Step(54, [3000, 5, 900, 64], [4, 1, 8, 2], hq=16, hk=2, dim=128)
    caches = s.device_caches()
    one = attention(s, caches)
    for _ in range(5):
        for a, b in zip(one, attention(s, caches)):
            assert torch.equal(a, b)


def test_other_stream_and_overlapping_calls():
    import speculative_decoding_verification_rejection_gb300 as sv

    steps = [Step(60 + i, [1500 + i, 40], [3, 2], hq=8, hk=2, dim=128) for i in range(4)]
    side = [torch.cuda.Stream() for _ in steps]
    on = [(cuda(s.q), *s.device_caches(), cuda(s.table), cuda(s.lengths), cuda(s.cu)) for s in steps]
    torch.cuda.synchronize()
    got = [sv.cache_attention(*a[:5], cu_num_draft=a[5], lse=True, stream=t) for _ in range(3) for a, t in zip(on, side)][-4:]
    with torch.cuda.stream(side[0]):
        inner = sv.cache_attention(*on[0][:5], cu_num_draft=on[0][5], lse=True)
    torch.cuda.synchronize()
    for s, g in zip(steps, got):
        want, err = ref_attention(s)
        for a, w, e in zip(g, want, err):
            off_by(a, w, e, "other stream")
    assert torch.equal(inner[0], got[0][0])


def test_captured_steps_follow_their_device_side_lengths():
    """Two graphs, each append and attention of one step, replayed in turn while the lengths grow."""
    import speculative_decoding_verification_rejection_gb300 as sv

    inv = cuda(freqs(32))
    held = []
    for seed in (70, 71):
        s = Step(seed, [900, 3, 64], [2, 1, 3], hq=8, hk=2, dim=64, spare=4)
        for i in range(s.n):   # pages for what is to come
            s.table[i] = (s.table[i] * 0 + torch.arange(s.width) + i * s.width).int()
        s.pool = s.n * s.width
        s.k_cache, s.v_cache = (torch.randn(s.pool, s.page, s.hk, s.dim).to(s.kind) for _ in range(2))
        k, v = s.device_caches()
        t = dict(q=cuda(s.q), k=cuda(s.k), v=cuda(s.v), kc=k, vc=v, table=cuda(s.table), lengths=cuda(s.lengths), cu=cuda(s.cu))

        def step(t=t):
            q = sv.cache_append(t["k"], t["v"], t["kc"], t["vc"], t["table"], t["lengths"], q=t["q"], inv_freq=inv, cu_num_draft=t["cu"])
            return q, *sv.cache_attention(q, t["kc"], t["vc"], t["table"], t["lengths"], cu_num_draft=t["cu"], lse=True)

        step()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        held.append((s, t, g, out))
    for grow in (0, 1, 17, 40):
        for s, t, g, out in held:
            s.lengths += grow
            t["lengths"] += grow
            g.replay()
        torch.cuda.synchronize()
        for s, t, g, out in held:
            want, err = ref_append(s, freqs(32))
            for name, got, w, e in zip("qkv", (out[0], t["kc"], t["vc"]), want, err):
                off_by(got, w, e, name)
            asked = s.q
            s.q, s.k_cache, s.v_cache = out[0].cpu(), t["kc"].cpu(), t["vc"].cpu()
            want, err = ref_attention(s)
            s.q = asked
            for name, got, w, e in zip(("out", "lse"), out[1:], want, err):
                off_by(got, w, e, name)


def test_captured_behind_copies_and_another_stream():
    """In a graph a call may follow a copy, a fill, a kernel, and work of another stream that is joined before it."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(75, [300, 20], [3, 2], hq=8, hk=2, dim=64, page=16)
    k, v = s.device_caches()
    table, lengths, cu, q0 = cuda(s.table), cuda(s.lengths), cuda(s.cu), cuda(s.q)
    q, ks, vs = torch.zeros_like(q0), torch.zeros_like(cuda(s.k)), cuda(s.v)
    kk = cuda(s.k)
    out, lse = torch.empty_like(q), torch.empty(s.rows, s.hq, device="cuda")
    side = torch.cuda.Stream()

    def step():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            ks.copy_(kk)
        q.zero_()
        here.wait_stream(side)
        sv.cache_append(ks, vs, k, v, table, lengths, cu_num_draft=cu)
        q.copy_(q0)
        sv.cache_attention(q, k, v, table, lengths, cu_num_draft=cu, lse=True, out=[out, lse])

    step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(3):
        out.fill_(9)
        k[s.slot(0, 300)] = 0
        g.replay()
    torch.cuda.synchronize()
    for r, i, x in s.rows_of():
        s.k_cache[s.slot(i, x)], s.v_cache[s.slot(i, x)] = s.k[r], s.v[r]
    want, err = ref_attention(s)
    off_by(out, want[0], err[0], "out")
    off_by(lse, want[1], err[1], "lse")


def test_an_empty_pool():
    """No page at all: nothing is written, no key is seen."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(76, [30, 2], [2, 3], hq=4, hk=2, dim=64)
    for kind in (torch.bfloat16, torch.float8_e4m3fn):
        none = torch.zeros(0, 16, 2, 64, dtype=kind, device="cuda")
        q = sv.cache_append(cuda(s.k), cuda(s.v), none, torch.zeros_like(none), cuda(s.table), cuda(s.lengths), q=cuda(s.q), cu_num_draft=cuda(s.cu))
        assert torch.equal(q, cuda(s.q))
        out, lse = sv.cache_attention(cuda(s.q), none, none, cuda(s.table), cuda(s.lengths), cu_num_draft=cuda(s.cu), lse=True)
        assert bool((out == 0).all()) and bool((lse == -float("inf")).all())


def test_offsets_beyond_32_bits():
    """A pool of 6 GB with the pages in use at its end."""
    import speculative_decoding_verification_rejection_gb300 as sv

    pages, page, hk, dim = 24000, 64, 8, 256
    k = torch.zeros(pages, hk, page, dim, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    v = torch.zeros(pages, hk, page, dim, dtype=torch.bfloat16, device="cuda").transpose(1, 2)
    s = Step(80, [150], [3], hq=8, hk=hk, dim=dim, page=page)
    used = s.width
    small_k, small_v = s.k_cache, s.v_cache
    at = [pages - 1 - 7 * c for c in range(used)]
    for c in range(used):
        k[at[c]] = small_k[s.table[0, c]].cuda()
        v[at[c]] = small_v[s.table[0, c]].cuda()
    table = torch.tensor([at], dtype=torch.int32, device="cuda")
    out, lse = sv.cache_attention(cuda(s.q), k, v, table, cuda(s.lengths), cu_num_draft=cuda(s.cu), lse=True)
    want, err = ref_attention(s)
    off_by(out, want[0], err[0], "out")
    off_by(lse, want[1], err[1], "lse")
    sv.cache_append(cuda(s.k), cuda(s.v), k, v, table, cuda(s.lengths), cu_num_draft=cuda(s.cu))
    for j in range(3):
        x = 150 + j
        assert torch.equal(k[at[x // page], x % page].cpu(), s.k[j]) and torch.equal(v[at[x // page], x % page].cpu(), s.v[j])
    assert int((k[:at[-1]] != 0).sum()) == 0


def test_parts_of_an_attention_join_by_their_lse():
    """The first tokens' pages and the others' attended in two calls, joined by the logarithms of their sums."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(81, [400, 250], [1, 1], hq=4, hk=2, dim=64, page=16)
    k, v = s.device_caches()
    whole = sv.cache_attention(cuda(s.q), k, v, cuda(s.table), cuda(s.lengths), lse=True)
    head = sv.cache_attention(cuda(s.q), k, v, cuda(s.table[:, :8].contiguous()), cuda(s.lengths), lse=True)   # 128 places
    rest = sv.cache_attention(cuda(s.q), k, v, cuda(s.table[:, 8:].contiguous()), cuda(s.lengths - 128), lse=True)
    top = torch.maximum(head[1], rest[1])
    a, b = torch.exp(head[1] - top), torch.exp(rest[1] - top)
    joined = (head[0].float() * a[..., None] + rest[0].float() * b[..., None]) / (a + b)[..., None]
    want, err = ref_attention(s)
    off_by(joined, want[0], 3 * err[0], "joined")      # (both parts rounded as the whole is)
    off_by(top + torch.log(a + b), want[1], 3 * err[1] + 1e-5, "joined lse")
    off_by(whole[0], want[0], err[0], "whole")


# --------------------------------------------------------------------------- run together

def test_steps_of_a_verification_over_the_cache():
    """A toy decoder of one layer: each step appends the rows of the last tokens and their drafts, attends, makes
    logits, verifies, and moves the lengths on by what was sampled. After some steps with rejections, one more
    attention over the cache equals that over the emitted sequence, computed without a cache in 64 bits."""
    import speculative_decoding_verification_rejection_gb300 as sv

    torch.manual_seed(5)
    n, K, vocab, hq, hk, dim, page = 5, 3, 97, 4, 2, 64, 16
    dev, bf = "cuda", torch.bfloat16
    embed = torch.randn(vocab, 64, device=dev).to(bf)
    w = {x: (torch.randn(64, h * dim, device=dev) / 8).to(bf) for x, h in (("q", hq), ("k", hk), ("v", hk))}
    head = (torch.randn(hq * dim, vocab, device=dev) / 16).to(bf)
    inv = cuda(freqs(dim // 2))
    width = 6
    kc, vc = (torch.zeros(n * width, page, hk, dim, dtype=bf, device=dev) for _ in range(2))
    table = torch.randperm(n * width).int().view(n, width).cuda()
    lengths = torch.zeros(n, dtype=torch.int32, device=dev)
    cu = torch.arange(n + 1, dtype=torch.int32, device=dev) * K
    ctx = sv.SpecVerify(n, K, vocab, "bf16", has_draft_probs=False)
    last = torch.randint(0, vocab, (n,), device=dev)
    history = [[int(t)] for t in last]
    g = torch.Generator(device=dev).manual_seed(6)
    rejected = 0
    for step in range(12):
        drafts = torch.randint(0, vocab, (n, K), device=dev, generator=g)
        tokens = torch.cat((last[:, None], drafts), 1).flatten()
        x = embed[tokens]
        q, k, v = ((x @ w[a]).view(n * (K + 1), -1, dim) for a in "qkv")
        q = sv.cache_append(k, v, kc, vc, table, lengths, q=q, inv_freq=inv, cu_num_draft=cu)
        out, = sv.cache_attention(q, kc, vc, table, lengths, cu_num_draft=cu)
        logits = (out.flatten(1) @ head).contiguous()
        if step % 3 == 0:    # some drafts that the target would choose itself
            drafts = logits.view(n, K + 1, vocab)[:, :K].argmax(-1)
            tokens = torch.cat((last[:, None], drafts), 1).flatten()
            x = embed[tokens]
            q, k, v = ((x @ w[a]).view(n * (K + 1), -1, dim) for a in "qkv")
            q = sv.cache_append(k, v, kc, vc, table, lengths, q=q, inv_freq=inv, cu_num_draft=cu)
            out, = sv.cache_attention(q, kc, vc, table, lengths, cu_num_draft=cu)
            logits = (out.flatten(1) @ head).contiguous()
        sampled, num, num_rejected = ctx.run(logits, drafts.int().flatten().contiguous(), None, cu, torch.ones(n, device=dev),
                                             torch.ones(n, dtype=torch.uint8, device=dev), seed=step)
        lengths += num
        last = sampled.gather(1, (num - 1).long()[:, None])[:, 0].long()
        rejected += int(num_rejected.sum())
        for i in range(n):
            history[i] += sampled[i, :int(num[i])].tolist()
    assert ctx.last_error() == 0 and rejected > 0
    ctx.close()
    assert [len(h) - 1 for h in history] == lengths.tolist()
    x = embed[last]
    q, k, v = ((x @ w[a]).view(n, -1, dim) for a in "qkv")
    q = sv.cache_append(k, v, kc, vc, table, lengths, q=q, inv_freq=inv)
    out, = sv.cache_attention(q, kc, vc, table, lengths)
    for i in range(n):
        x = embed[torch.tensor(history[i], device=dev)]
        kk, vv = ((x @ w[a]).view(-1, hk, dim).double() for a in "kv")
        angle = torch.arange(len(history[i]), device=dev)[:, None].double() * inv.double()
        c, s_ = angle.cos()[:, None], angle.sin()[:, None]
        one, two = kk[..., :32], kk[..., 32:]
        kk = torch.cat((one * c - two * s_, one * s_ + two * c), -1)
        for h in range(hq):
            score = kk[:, h // 2] @ q[i, h].double() / 8
            want = torch.softmax(score, 0) @ vv[:, h // 2]
            # keys rounded to bf16 (2^-8 of a score's terms), weights and the output besides
            size = (kk[:, h // 2].abs() @ q[i, h].double().abs() / 8).max() * 2.0**-8
            tol = float(vv[:, h // 2].abs().max()) * (2 * float(size) + 3 * 2.0**-8)
            assert float((out[i, h].double() - want).abs().max()) <= tol


def test_overlapping_requests_of_too_many_tiles_are_left_out():
    """Prefix sums that are none, by which 1000 requests have the same 2000 rows: 4.4e9 tiles of keys, which no 32 bits
    hold (the rows that there are have 78 million at most)."""
    import speculative_decoding_verification_rejection_gb300 as sv

    n, page, width = 2000, 65536, 34
    pool = torch.zeros(1, page, 2, 64, dtype=torch.bfloat16, device="cuda")
    table = torch.zeros(n, width, dtype=torch.int32, device="cuda")
    lengths = torch.full((n,), page * width - 10, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 2000] * (n // 2) + [0], dtype=torch.int32, device="cuda")
    q = torch.zeros(4100, 2, 64, dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((4100, 2), 7.0, device="cuda")
    sv.cache_attention(q, pool, pool, table, lengths, cu_num_draft=cu, lse=True, out=[out, lse])
    torch.cuda.synchronize()
    assert bool((out == 7).all()) and bool((lse == 7).all())
    # the same arrays with lengths that 32 bits hold
    lengths.fill_(0)
    sv.cache_attention(q, pool, pool, table, lengths, cu_num_draft=cu, lse=True, out=[out, lse])
    assert bool((out[:2001] == 0).all()) and bool((out[4000:] == 7).all())


@pytest.mark.parametrize("cache", ("bf16", "e4m3"))
def test_steps_right_behind_what_writes_their_inputs(cache):
    """Lengths, prefix sums and pages moved on by small kernels, queries turned in place, and their attention, one right behind the
    other: as with a wait for the device after each."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(90, [700, 3, 64, 1500], [2, 1, 3, 2], hq=8, hk=2, dim=128, cache=cache, page=16, layout="heads", spare=8)
    inv = cuda(freqs(64))
    g = torch.Generator(device="cuda").manual_seed(7)
    rows = torch.randn(40, 3, s.rows, s.hq, s.dim, generator=g, device="cuda").to(s.dtype)
    tables = torch.stack([torch.randperm(s.n * s.width, generator=g, device="cuda").view(s.n, s.width) for _ in range(40)]).int()
    sums = torch.stack((cuda(s.cu), torch.tensor([0, 0, 2, 3, 4], device="cuda"))).int()

    def steps(wait):
        pool = torch.zeros(s.n * s.width, s.page, s.hk, s.dim, device="cuda").to(s.kind)
        k, v = pool, pool.clone()
        lengths, table, cu = cuda(s.lengths), tables[0].clone(), sums[0].clone()
        q, kk, vv = (torch.empty_like(rows[0, 0]) for _ in range(3))
        got = []
        for t in range(40):
            for to, x in ((q, rows[t, 0]), (kk, rows[t, 1]), (vv, rows[t, 2]), (table, tables[t // 8]), (cu, sums[t % 2])):
                to.copy_(x)
                wait()
            lengths.add_(1)
            wait()
            sv.cache_append(kk[:, :s.hk], vv[:, :s.hk], k, v, table, lengths, q=q, inv_freq=inv, cu_num_draft=cu, out=q)
            wait()
            got.append((q.clone(), *sv.cache_attention(q, k, v, table, lengths, cu_num_draft=cu, lse=True)))
            wait()
        return [x for step in got for x in step] + [k.view(torch.uint8), v.view(torch.uint8)]

    want = steps(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(steps(lambda: None), want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("scale", (7 / 512, 13 / 512, 15 / 512, 61 / 512, 1.0, 0.75, 3e-3, -0.25, 2.0**-140, 1e30,
                                   0.0371, -7 / 512, 1.7 * 2.0**99, 1.2 * 2.0**100, 1.3 * 2.0**-100, 1.7 * 2.0**-101, 2.0**-126, 2.0**126))
def test_append_8_bits_divides_by_the_scale(scale):
    """Every bfloat16 number as a value: what is stored is its quotient by the scale, rounded to 8 bits (with 7, 13, 15 and 61 / 512
    some quotients are ties, which a product with the reciprocal misses; 2^-140 has no reciprocal)."""
    import speculative_decoding_verification_rejection_gb300 as sv

    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).view(32, 8, 256)
    v = torch.where(torch.isnan(v), torch.zeros(()).bfloat16(), v)
    by = torch.full((8,), scale)
    k_cache, v_cache = (torch.zeros(4, 16, 8, 256, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2))
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    sv.cache_append(cuda(v), cuda(v), k_cache, v_cache, table, torch.zeros(1, dtype=torch.int32, device="cuda"),
                    cu_num_draft=torch.tensor([0, 31], dtype=torch.int32, device="cuda"), k_scale=cuda(by), v_scale=cuda(by))
    want = (v.float() / by[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    for cache in (k_cache, v_cache):   # (without frequencies nothing is turned)
        assert torch.equal(torch.cat((cache[2], cache[0])).cpu().view(torch.uint8), want)


@pytest.mark.parametrize("group", (2, 16))
@pytest.mark.parametrize("cache,size,scale", (("bf16", 2.0**60, 1.0), ("bf16", 2.0**60, 2.0**-126), ("e4m3", 2.0**110, 512.0)))
def test_a_first_key_far_below_after_tiles_without_one(cache, size, scale, group):
    """The keys of the first tiles are not there (bad pages); the first that is has a score of -2^126 (or, as little, -1). With 16 query
    heads to a key head the rows of a tile are all queries (others' scores of 0 would set a reference)."""
    import speculative_decoding_verification_rejection_gb300 as sv

    n, page, hk, dim, length = 64, 16, 2, 64, 600
    g = torch.Generator(device="cuda").manual_seed(3)
    key = 1.0 if cache == "e4m3" else size
    k = torch.full((n, page, hk, dim), key, device="cuda").to(TYPES[cache])
    v = torch.randn(n, page, hk, dim, generator=g, device="cuda").to(TYPES[cache])
    table = torch.full((n, length // page + 1), -1, dtype=torch.int32, device="cuda")
    table[:, -1] = torch.arange(n, device="cuda")
    q = torch.full((n, group * hk, dim), -size, device="cuda").bfloat16()
    out, lse = sv.cache_attention(q, k, v, table, torch.full((n,), length, dtype=torch.int32, device="cuda"), scale=scale, lse=True)
    seen = length % page + 1      # all of the same score: their mean, each weight exactly 1
    score = -size * key * dim * scale
    mean = v[:, :seen].double().mean(1).repeat_interleave(group, 1)
    # the output's rounding to bfloat16 (8 significant bits: half a step is 2^-8 of the value at most), on top of sums of nine terms below 5 in binary32
    assert bool(((out.double() - mean).abs() <= mean.abs() * 2.0**-8 + 2.0**-18).all())
    want = score + math.log(seen)
    assert float((lse.double() - want).abs().max()) <= abs(want) * 2.0**-21


@pytest.mark.parametrize("page", (7, 8, 9, 11, 14, 15, 37, 111, 112, 125, 130, 223, 224, 249, 255, 500))
@pytest.mark.parametrize("dim,cache", ((64, "bf16"), (128, "f16"), (256, "bf16"), (64, "e4m3"), (128, "e4m3"), (256, "e4m3")))
def test_attention_pages_beside_the_border_of_the_two_ways_to_copy(page, dim, cache):
    """Pages that just fill, or do not fill, seven eighths of a tile, in one part or several, and the smallest that tensor maps bring."""
    dtype = "bf16" if cache == "e4m3" else cache
    s = Step(page + dim, LENGTHS + [page * 2 - 1, 1300], NEW + [2, 5], hq=6, hk=2, dim=dim, dtype=dtype, cache=cache, page=page, layout="heads", spare=1)
    check_attention(s)
    check_attention(s, window=150)


def long_runs(dim, hq, cache, page, whole):
    """96 requests of 4 rows over up to 3100 keys (14 of them over fewer than 14) in pages that requests share: arguments of a call,
    and keys and values as the requests see them, in 64 bits. `whole`: values are whole numbers from -8 to 8."""
    n, width, new = 96, 3200 // page, 4
    g = torch.Generator(device="cuda").manual_seed(dim + hq + page)
    k = torch.randn(300, page, 1, dim, generator=g, device="cuda").to(TYPES[cache])
    v = (torch.randint(-8, 9, k.shape, generator=g, device="cuda") if whole else torch.randn(k.shape, generator=g, device="cuda")).to(TYPES[cache])
    table = torch.randint(0, 300, (n, width), generator=g, device="cuda").int()
    lengths = torch.randint(0, 3100, (n,), generator=g, device="cuda").int()
    lengths[::7] = torch.arange(14, device="cuda").int()
    q = torch.randn(n * new, hq, dim, generator=g, device="cuda").bfloat16()
    keys, values = (c[table.long()].float().view(n, -1, dim).double() for c in (k, v))
    seen = torch.arange(width * page, device="cuda") <= lengths[:, None, None].long() + torch.arange(new, device="cuda")[:, None]
    return (q, k, v, table, lengths), dict(cu_num_draft=torch.arange(n + 1, device="cuda").int() * (new - 1), lse=True), keys, values, seen


RUNS = pytest.mark.parametrize("dim,hq", ((256, 8), (256, 16), (128, 8), (128, 12), (128, 16), (64, 24)))
WAYS = pytest.mark.parametrize("cache,page", (("bf16", 32), ("e4m3", 32), ("bf16", 4), ("e4m3", 4)))


@RUNS
@WAYS
def test_every_value_of_long_runs_of_tiles_counts_once(dim, hq, cache, page):
    """With a scale of 0 every weight is the same power of two and sums of whole numbers are exact: an output is the mean of the values
    but for a division and its rounding, and one value too many, too few or of another tile shows (by 1 / 3100 of a unit or more)."""
    import speculative_decoding_verification_rejection_gb300 as sv

    args, kw, _, values, seen = long_runs(dim, hq, cache, page, whole=True)
    out, lse = sv.cache_attention(*args, scale=0.0, **kw)
    count = seen.sum(-1)
    want = (torch.einsum("nrt,ntd->nrd", seen.double(), values) / count[..., None])[:, :, None]
    off = (out.view(96, 4, hq, dim).double() - want).abs()
    # half a step of bfloat16, and a quotient and a product in binary32 before it
    assert bool((off <= want.abs() * (2.0**-8 + 2.0**-21)).all())
    assert float((lse.view(96, 4, hq).double() - count.double().log()[..., None]).abs().max()) <= 2.0**-19   # (log2 and a product, of numbers up to 12)


@RUNS
@WAYS
def test_long_runs_of_tiles_element_by_element(dim, hq, cache, page):
    """Every output within what its own weights' and scores' roundings allow, and three calls alike bit for bit."""
    import speculative_decoding_verification_rejection_gb300 as sv

    args, kw, keys, values, seen = long_runs(dim, hq, cache, page, whole=False)
    out, lse = sv.cache_attention(*args, **kw)
    for _ in range(2):
        again = sv.cache_attention(*args, **kw)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)
    q = args[0].view(96, 4, hq, dim).double()
    weight = 2.0**-8 if cache == "bf16" else 2.0**-11
    many = (3200 / 8 + 32) * 2.0**-22
    for i in range(96):
        score = (q[i] @ keys[i].T * dim ** -0.5).masked_fill(~seen[i][:, None], -float("inf"))
        p = torch.softmax(score, -1)
        want, size, z = p @ values[i], p @ values[i].abs(), torch.logsumexp(score, -1)
        # as in tests/_cache.py: a score's products added in units that may cut, its factor, the argument of 2^x; and its use in numerator and sum
        terms = (q[i].abs() @ keys[i].abs().T).masked_fill(~seen[i][:, None], 0)
        away = (terms * (dim * 2.0**-22) + (q[i].abs().amax(-1, keepdim=True) * keys[i].abs().sum(-1)).masked_fill(~seen[i][:, None], 0) * 2.0**-35).amax(-1) * dim ** -0.5
        away = away + 3 * 2.0**-24 * torch.where(torch.isfinite(score), score.abs(), 0).amax(-1) + 2.0**-22
        allowed = size * (weight + 2 * away[..., None] + 2 * many) * 1.01 + want.abs() * 2.0**-8 * 1.01
        allowed = allowed + (seen[i].double() @ values[i].abs())[:, None] * 2.0**-36 * p.amax(-1, keepdim=True)
        off = (out.view(96, 4, hq, dim)[i].double() - want).abs()
        assert bool((off <= allowed).all()), f"request {i}: {float((off / allowed).max())} of the bound"
        assert bool(((lse.view(96, 4, hq)[i].double() - z).abs() <= away + many + 2.0**-22 * z.abs()).all())


@pytest.mark.parametrize("cu", ([0, 1, 0, 5], [0, -3, 2, 5], [0, 2, 2**31 - 1, 5], [-2**31, 0, 1, 2], [0, 100, 100, 100], [7, 7, 7, 7]))
def test_requests_that_inconsistent_prefix_sums_leave_are_right(cu):
    """The requests whose rows are all within the batch are appended and attended for; nothing is written for other rows."""
    import speculative_decoding_verification_rejection_gb300 as sv

    s = Step(53, [10, 20, 30], [2, 1, 5], dim=64, spare=1)
    s.table = torch.arange(s.n * s.width).int().view(s.n, s.width)
    s.pool = s.n * s.width
    g = torch.Generator().manual_seed(1)
    s.k_cache, s.v_cache = (torch.randn(s.pool, s.page, s.hk, s.dim, generator=g).to(s.kind) for _ in range(2))
    rows = s.rows
    for i in range(s.n):
        first, count = cu[i] + i, cu[i + 1] - cu[i] + 1
        s.first[i], s.new[i] = first, count if cu[i] >= 0 and count >= 1 and first + count <= rows else 0
    valid = [r for r, _, _ in s.rows_of()]
    assert len(valid) == len(set(valid))
    k, v = s.device_caches()
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    q = torch.full((rows, s.hq, s.dim), 5.0, dtype=s.dtype, device="cuda")
    out, lse = torch.full_like(q, 5.0), torch.full((rows, s.hq), 5.0, device="cuda")
    sv.cache_append(cuda(s.k), cuda(s.v), k, v, cuda(s.table), cuda(s.lengths), q=cuda(s.q), inv_freq=cuda(freqs(32)), cu_num_draft=bad, out=q)
    others = [r for r in range(rows) if r not in valid]
    (want_q, want_k, want_v), (qe, ke, ve) = ref_append(s, freqs(32))
    off_by(k, want_k, ke, "k")     # (slots of no valid row as they were)
    off_by(v, want_v, ve, "v")
    off_by(q[valid], want_q[valid], qe[valid], "q")
    assert bool((q[others] == 5).all())
    s.k_cache, s.v_cache = k.cpu(), v.cpu()
    sv.cache_attention(cuda(s.q), k, v, cuda(s.table), cuda(s.lengths), cu_num_draft=bad, lse=True, out=[out, lse])
    (want, want_lse), (oe, le) = ref_attention(s)
    off_by(out[valid], want[valid], oe[valid], "out")
    off_by(lse[valid], want_lse[valid], le[valid], "lse")
    assert bool((out[others] == 5).all()) and bool((lse[others] == 5).all())
