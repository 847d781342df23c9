"""The 4-bit K/V cache on the GPU: what is written and read back, bit for bit,
and attention over it within the derived bounds of tests/cache_ref.py, at the
sizes, layouts and masks where they can go wrong; graphs, streams, bad indices
and the run of a prompt, a chunk and single tokens as a server makes it."""
import numpy as np
import pytest
import torch

import cache_ref
from exact_io_aware_attention_gb300 import binding
from exact_io_aware_attention_gb300 import inputs as gen

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16
BAD_INDEX = 0xC0000000


def fa():
    import exact_io_aware_attention_gb300 as m
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rand(shape, seed, dtype):
    return gen.normal_bf16(shape, seed, dtype)


def random_table(B, pages, seed, spare=3):
    """[B, pages] distinct pages of a pool with `spare` more."""
    g = torch.Generator().manual_seed(seed)
    n = B * pages + spare
    return torch.randperm(n, generator=g)[:B * pages].reshape(B, pages).to(torch.int32), n


def widen(table, page):
    """The table with room for more than 1024 tokens, beyond which sequences are split between
    CTAs and 65 rows a K/V head count as many. What the new entries say is never read."""
    return torch.cat([table, torch.full((table.shape[0], 1024 // page + 1), 1 << 30,
                                        dtype=torch.int32, device=table.device)], 1)


def new_cache(n_pages, H, d, page, dtype, fill=0xFF):
    """A cache whose untouched groups read as NaN."""
    c = fa().KVCache4(n_pages, H, d, page_size=page, dtype=dtype)
    c.data.fill_(fill)
    return c


def same_bits(a, b):
    a, b = a.cpu(), b.cpu()
    return a.dtype == b.dtype and torch.equal(torch.isnan(a), torch.isnan(b)) and \
        torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def clean():
    torch.cuda.synchronize()
    assert fa().device_status() == 0


# ------------------------------------------------------------------ write and read

@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,H,n,page,start", [
    (1, 1, 1, 16, [0]),
    (3, 2, 37, 16, [0, 5, 90]),       # pages that end inside the rows, odd starts
    (2, 5, 130, 48, [47, 1]),         # a page size that is no power of two
    (4, 3, 3, 64, [61, 62, 63, 64]),  # over a page's end and at it
    (1, 2, 300, 256, [17]),
])
def test_rows_come_back_as_the_formula_says(d, dtype, B, H, n, page, start):
    k, v = rand((B, H, n, d), 1, dtype), rand((B, H, n, d), 2, dtype) * 0.01 + 1
    table, pool = random_table(B, -(-(max(start) + n) // page), seed=d)
    c = new_cache(pool, H, d, page, dtype)
    fa().cache_write(c, k.cuda(), v.cuda(), table.cuda(), ints(start))
    k2, v2 = fa().cache_read(c, table.cuda(), ints(start), n)
    clean()
    assert torch.equal(k2.cpu(), cache_ref.read_back(k))
    assert torch.equal(v2.cpu(), cache_ref.read_back(v))


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_values_where_quantisers_go_wrong(d, dtype):
    big = 6e4 if dtype == F16 else 2e38
    tiny = torch.finfo(dtype).smallest_normal
    x = rand((1, 1, 64, d), 3, dtype)
    x[0, 0, 0] = 0.0
    x[0, 0, 1] = -0.0
    x[0, 0, 2] = 2.5                                        # s = 0
    x[0, 0, 3] = big
    x[0, 0, 4, 0::2], x[0, 0, 4, 1::2] = big, -big          # bf16: the range overflows
    x[0, 0, 5, 7], x[0, 0, 6, 40], x[0, 0, 7, 63] = float("nan"), float("inf"), -float("inf")
    x[0, 0, 8] = torch.arange(d).to(dtype) % 31 * 0.5        # ties of (x - lo) / s
    x[0, 0, 9] = (torch.arange(d).to(dtype) % 16) * tiny     # steps of one subnormal
    x[0, 0, 10] = (torch.arange(d).to(dtype) % 3) * (tiny * torch.finfo(dtype).eps)  # s = 0
    x[0, 0, 11] = 1000 + torch.arange(d).to(dtype) % 32      # an offset far above the range
    x[0, 0, 12] = -x[0, 0, 11]
    x[0, 0, 13, :32] = 1e-3 * x[0, 0, 20, :32]
    table = ints([[0]])
    c = new_cache(1, 1, d, 64, dtype)
    fa().cache_write(c, x.cuda(), x.flip(2).cuda(), table, ints([0]))
    k2, v2 = fa().cache_read(c, table, ints([0]), 64)
    clean()
    assert same_bits(k2, cache_ref.read_back(x))
    assert same_bits(v2, cache_ref.read_back(x.flip(2)))


@pytest.mark.parametrize("d,dtype", [(64, BF16), (96, F16), (128, F16), (256, BF16)])
def test_strided_rows_counts_and_neighbours(d, dtype):
    """[B, N, H, d] rows, a table that is a view, ragged counts; tokens that no row is for, and
    rows of the outputs that no token is for."""
    B, H, n, page = 4, 3, 21, 32
    k = rand((B, n, H, d), 11, dtype).permute(0, 2, 1, 3)
    v = rand((B, n, 2 * H, d), 12, dtype).cuda()[:, :, ::2].permute(0, 2, 1, 3)
    old_k, old_v = rand((B, H, 2 * page, d), 13, dtype), rand((B, H, 2 * page, d), 14, dtype)
    table, pool = random_table(B, 5, seed=9)
    table = table.cuda()[:, 1:3]  # row stride 5, two pages a row
    c = new_cache(pool, H, d, page, dtype)
    fa().cache_write(c, old_k.cuda(), old_v.cuda(), table, ints([0] * B))
    before = c.data.clone()
    start, counts = [0, 30, 43, 5], [21, 0, 20, 1]
    fa().cache_write(c, k.cuda(), v, table, ints(start), ints(counts))
    out_k = torch.full((B, 2 * page, H, d), 7.0, dtype=dtype, device="cuda").permute(0, 2, 1, 3)
    fa().cache_read(c, table, ints([0] * B), 2 * page, ints([64, 64, 63, 64]), k=out_k)
    k2, v2 = fa().cache_read(c, table, ints([0] * B), 2 * page, ints([64, 64, 63, 64]))
    clean()
    assert torch.equal(k2, out_k)
    for b in range(B):
        for got, old, new in ((k2, old_k, k), (v2, old_v, v.cpu())):
            want = cache_ref.read_back(old[b])
            want[:, start[b]:start[b] + counts[b]] = cache_ref.read_back(new[b, :, :counts[b]])
            if b == 2:
                want[:, 63:] = 0
            assert torch.equal(got[b].cpu(), want), b
    # pages of no sequence stay as they were
    cells = c.data.reshape(pool, -1)
    mine = set(table.flatten().tolist())
    rest = [p for p in range(pool) if p not in mine]
    assert torch.equal(cells[rest], before.reshape(pool, -1)[rest])


def test_pool_beyond_32_bit_offsets():
    """Pages whose bytes lie past 4 GiB of the pool."""
    d, page, H = 128, 64, 1
    per_page = 64 * 320
    pool = (1 << 32) // per_page + 5
    c = fa().KVCache4(pool, H, d, page_size=page)
    table = ints([[pool - 1, 0, pool - 3]])
    k, v = rand((1, H, 150, d), 21, BF16), rand((1, H, 150, d), 22, BF16)
    fa().cache_write(c, k.cuda(), v.cuda(), table, ints([0]))
    k2, v2 = fa().cache_read(c, table, ints([0]), 150)
    q = rand((1, 2, 1, d), 23, BF16)
    o, lse = fa().cache_forward(q.cuda(), c, table, ints([150]), causal=True)
    clean()
    assert torch.equal(k2.cpu(), cache_ref.read_back(k))
    assert torch.equal(v2.cpu(), cache_ref.read_back(v))
    compare(o, lse, q, k, v, [150], None, True, None, "past 4 GiB")


# ------------------------------------------------------------------ attention

def compare(o, lse, q, k, v, lengths, counts, causal, scale, what):
    """O and LSE of a call against the plain implementation within its bounds."""
    B, Hq, Nq, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    eps = torch.finfo(o.dtype).eps
    for b in range(B):
        n = Nq if counts is None else counts[b]
        L = lengths[b]
        ro, rl, to, tl = cache_ref.attend(q[b], k[b, :, :L], v[b, :, :L], n, causal, scale, eps)
        go, gl = o[b].cpu().double().numpy(), lse[b].cpu().double().numpy()
        none = np.isneginf(rl)
        assert (np.isneginf(gl) == none).all(), (what, b)
        assert (go[none] == 0).all(), (what, b)
        err = np.abs(go - ro)
        assert (err <= to).all(), (what, b, float((err / np.maximum(to, 1e-300)).max()))
        el = np.abs(gl[~none] - rl[~none])
        assert (el <= tl[~none]).all(), (what, b, float((el / tl[~none]).max(initial=0)))


def attend_case(B, Hq, Hk, Nq, lengths, d, page, dtype, causal, counts=None, scale=None, o32=True,
                v_scale=1.0, k_scale=1.0, wide=False, what=""):
    L = max(lengths)
    k = (rand((B, Hk, max(L, 1), d), 31, dtype).float() * k_scale +
         rand((1, Hk, 1, d), 32, dtype).float() * k_scale).to(dtype)
    v = (rand((B, Hk, max(L, 1), d), 33, dtype).float() * v_scale).to(dtype)
    q = rand((B, Hq, Nq, d), 34, dtype)
    table, pool = random_table(B, max(1, -(-L // page)), seed=Nq + d)
    if wide:
        table = widen(table, page)
    c = new_cache(pool, Hk, d, page, dtype)
    fa().cache_write(c, k.cuda(), v.cuda(), table.cuda(), ints([0] * B), ints(lengths))
    cnt = None if counts is None else ints(counts)
    outs = []
    for dt in ([torch.float32, None] if o32 else [None]):
        outs.append(fa().cache_forward(q.cuda(), c, table.cuda(), ints(lengths), causal=causal,
                                       scale=scale, counts=cnt, o_dtype=dt))
    clean()
    for o, lse in outs:
        compare(o, lse, q, k, v, lengths, counts, causal, scale, what)
    return c, table, q, k, v


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("B,Hq,Hk,Nq,lengths,page", [
    (1, 1, 1, 1, [1], 16),
    (3, 4, 4, 1, [16, 17, 15], 16),
    (2, 8, 1, 1, [300, 63], 48),             # one group of eight heads
    (4, 6, 2, 3, [3, 200, 64, 129], 64),     # more rows than one 8-row tile
    (1, 5, 5, 2, [1500], 128),
    (2, 10, 2, 7, [40, 7], 32),              # 35 rows a K/V head, a partial tile
])
def test_attention_sizes(d, dtype, causal, B, Hq, Hk, Nq, lengths, page):
    attend_case(B, Hq, Hk, Nq, lengths, d, page, dtype, causal,
                what=f"{d} {dtype} {causal} {lengths}")


@pytest.mark.parametrize("d,dtype", [(64, BF16), (96, F16), (128, BF16), (256, F16)])
def test_rows_that_see_nothing(d, dtype):
    """Empty sequences, more new tokens than tokens, padded rows of a ragged batch."""
    attend_case(6, 4, 2, 5, [0, 2, 5, 100, 33, 0], d, 16, dtype, True, counts=[0, 5, 3, 0, 1, 5],
                what="counts")
    attend_case(6, 4, 2, 5, [0, 2, 5, 100, 33, 0], d, 16, dtype, False, counts=[0, 5, 3, 0, 1, 5],
                what="counts, not causal")


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("Nq,Hq,Hk", [(130, 2, 1), (33, 4, 2), (257, 1, 1)])
def test_chunks_of_a_prompt(d, Nq, Hq, Hk):
    attend_case(2, Hq, Hk, Nq, [Nq, Nq + 500], d, 64, BF16, True, o32=False, wide=True,
                what="chunk")
    attend_case(2, Hq, Hk, Nq, [Nq + 77, Nq], d, 32, F16, True, counts=[Nq - 5, Nq], what="chunk f16")


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("B,Hq,Hk,Nq,lengths,page,counts", [
    (1, 65, 1, 1, [1], 16, None),                       # one token, 65 heads on one
    (2, 24, 1, 3, [5, 200], 48, [3, 0]),                # 72 rows, an empty sequence of a batch
    (3, 20, 2, 40, [40, 300, 10], 16, [40, 7, 39]),     # 400 rows; more new tokens than tokens
    (1, 4, 1, 32, [1400], 128, None),                   # 128 rows; split between CTAs
    (2, 3, 1, 50, [129, 128], 64, None),                # tiles of 128 keys that end and begin
    (1, 6, 3, 150, [2000], 80, None),
    (1, 3, 1, 43, [2600], 64, None),                    # 129 rows: the second 128 hold one
    (5, 3, 1, 100, [1300, 128, 127, 700, 100], 32, None),  # pieces that begin at odd tiles
])
def test_many_rows(d, dtype, B, Hq, Hk, Nq, lengths, page, counts):
    for causal, wide in ((True, True), (False, True), (True, False)):
        attend_case(B, Hq, Hk, Nq, lengths, d, page, dtype, causal, counts=counts, wide=wide,
                    what=f"{d} {dtype} {causal} {wide} {lengths}")


@pytest.mark.parametrize("d", [64, 128])
def test_row_blocks_of_different_heights(d):
    """260 rows a K/V head are 256 and 4: CTAs walk over both kinds, at odd and even tiles."""
    B, Hk, Nq = 24, 8, 130
    lengths = [130 + (i * 97) % 400 for i in range(B)]
    table, pool = random_table(B, max(lengths) // 32 + 1, seed=7)
    table = widen(table, 32)
    k, v = rand((B, Hk, max(lengths), d), 151, BF16), rand((B, Hk, max(lengths), d), 152, BF16)
    q = rand((B, 2 * Hk, Nq, d), 153, BF16)
    c = new_cache(pool, Hk, d, 32, BF16)
    fa().cache_write(c, k.cuda(), v.cuda(), table.cuda(), ints([0] * B), ints(lengths))
    o, lse = fa().cache_forward(q.cuda(), c, table.cuda(), ints(lengths), causal=True)
    clean()
    for b in (0, 11, 23):
        compare(o[b:b + 1, :4], lse[b:b + 1, :4], q[b:b + 1, :4], k[b:b + 1, :2], v[b:b + 1, :2],
                lengths[b:b + 1], None, True, None, b)


@pytest.mark.parametrize("d,dtype,B", [(64, F16, 7), (64, BF16, 10), (96, BF16, 7), (128, F16, 10),
                                       (128, BF16, 7), (256, BF16, 7)])
def test_many_rows_of_short_sequences(d, dtype, B):
    """So many that they do not all run at once with few rows a CTA."""
    lengths = [(i * 53) % 190 for i in range(B)]
    attend_case(B, 8, 8, 150, lengths, d, 32, dtype, True, counts=[min(150, n) for n in lengths],
                o32=False, what="short")


@pytest.mark.parametrize("v_scale,k_scale", [(1e-3, 1.0), (300.0, 1.0), (1e-30, 1.0), (1e25, 1.0),
                                             (1.0, 30.0), (1.0, 1e-20)])
def test_sizes_of_values(v_scale, k_scale):
    """V far from 1 (the weights p s must keep their bits), sharp and flat scores."""
    attend_case(2, 4, 2, 2, [333, 40], 128, 32, BF16, True, v_scale=v_scale, k_scale=k_scale)
    attend_case(1, 40, 1, 2, [333], 128, 32, BF16, True, v_scale=v_scale, k_scale=k_scale,
                wide=True)
    attend_case(1, 40, 1, 2, [333], 256, 32, BF16, True, v_scale=v_scale, k_scale=k_scale,
                wide=True)
    if 1e-4 < v_scale < 1e3 and k_scale > 1e-4:
        attend_case(2, 4, 2, 2, [333, 40], 64, 32, F16, True, v_scale=v_scale, k_scale=k_scale)


def test_values_that_differ_by_magnitudes_between_tokens():
    """A first token with the score of a sink and a constant value (s = 0), others around it."""
    d, L = 64, 500
    k, v = rand((1, 1, L, d), 41, BF16), rand((1, 1, L, d), 42, BF16)
    q = rand((1, 2, 1, d), 43, BF16)
    k[0, 0, 0] = q[0, 0, 0] * 1.5
    v[0, 0, 0] = 0.0
    v[0, 0, 100:200] = (v[0, 0, 100:200].float() * 1e-6).to(BF16)
    v[0, 0, 300] = (v[0, 0, 300].float() * 1e4).to(BF16)
    table = ints([[2, 0, 3, 1, 5, 4, 6, 7]])
    c = new_cache(8, 1, d, 64, BF16)
    fa().cache_write(c, k.cuda(), v.cuda(), table, ints([0]))
    o, lse = fa().cache_forward(q.cuda(), c, table, ints([L]), o_dtype=torch.float32)
    clean()
    compare(o, lse, q, k, v, [L], None, False, None, "magnitudes")


def test_long_context_and_scale():
    attend_case(1, 2, 1, 1, [65536], 64, 64, BF16, True, scale=0.31, what="64k")
    attend_case(2, 4, 1, 2, [20001, 7], 128, 256, F16, True, scale=0.02, what="20k")


def test_one_warp_over_a_long_context():
    """Many sequences, so that one CTA walks a whole one: sums of thousands of products."""
    B, L, d = 700, 4096, 64
    k = rand((1, 1, L, d), 51, BF16).expand(B, 1, L, d)
    v = rand((1, 1, L, d), 52, BF16).expand(B, 1, L, d)
    q = rand((B, 1, 1, d), 53, BF16)
    c = new_cache(L // 64, 1, d, 64, BF16)
    one = torch.arange(L // 64, dtype=torch.int32, device="cuda")[None]
    fa().cache_write(c, k[:1].cuda(), v[:1].cuda(), one, ints([0]))
    table = one.expand(B, -1)  # every sequence reads the same pages: row stride 0
    o, lse = fa().cache_forward(q.cuda(), c, table, ints([L] * B), o_dtype=torch.float32)
    clean()
    for b in range(0, B, 97):
        compare(o[b:b + 1], lse[b:b + 1], q[b:b + 1], k[b:b + 1], v[b:b + 1], [L], None, False,
                None, b)


def test_many_short_sequences():
    """More blocks than threads look through at a time, with empty ones among them."""
    B = 300
    lengths = [(i * 37) % 90 for i in range(B)]
    attend_case(B, 4, 2, 1, lengths, 64, 16, BF16, True, o32=False, what="many")


def test_strided_queries_and_outputs():
    B, Hq, Hk, Nq, d = 2, 6, 3, 4, 96
    lengths = [100, 41]
    c, table, _, k, v = attend_case(B, Hq, Hk, Nq, lengths, d, 32, F16, True)
    q = rand((B, Nq, Hq, d), 61, F16)
    out = torch.full((B, Nq, 2 * Hq, d), 3.0, dtype=F16, device="cuda")
    view = out[:, :, ::2].permute(0, 2, 1, 3)
    o, lse = fa().cache_forward(q.cuda().permute(0, 2, 1, 3), c, table.cuda(), ints(lengths),
                                causal=True, out=view)
    clean()
    assert o is view and (out[:, :, 1::2] == 3.0).all()
    compare(o, lse, q.permute(0, 2, 1, 3), k, v, lengths, None, True, None, "strided")


@pytest.mark.parametrize("d,Hq", [(64, 2), (96, 2), (128, 2), (256, 2), (64, 17), (96, 20),
                                  (128, 36), (256, 20)])
def test_non_finite_values_stay_where_they_are_seen(d, Hq):
    """NaN and infinities in a key or value reach only the rows that see it, and only its
    group's outputs where it is a value; a NaN query spoils its own row alone."""
    B, Nq, L = 1, 4, 40
    k, v, q = (rand(s, 70 + i, BF16) for i, s in
               enumerate(((B, 1, L, d), (B, 1, L, d), (B, Hq, Nq, d))))
    table = ints([[1, 0, 2]])
    if Hq > 2:
        table = widen(table, 16)

    def run(k, v, q):
        c = new_cache(3, 1, d, 16, BF16)
        fa().cache_write(c, k.cuda(), v.cuda(), table, ints([0]))
        o, lse = fa().cache_forward(q.cuda(), c, table, ints([L]), causal=True)
        clean()
        return o.cpu(), lse.cpu()

    good_o, good_lse = run(k, v, q)
    for bad in (float("nan"), float("inf")):
        v1 = v.clone()
        v1[0, 0, L - 2, 5] = bad      # seen by the last two rows
        o, lse = run(k, v1, q)
        assert torch.equal(o[:, :, :2], good_o[:, :, :2]) and torch.equal(lse, good_lse)
        assert torch.isnan(o[:, :, 2:, :32]).all()
        assert not torch.isnan(o[:, :, 2:, 32:]).any()
        k1 = k.clone()
        k1[0, 0, L - 1, 9] = bad      # seen by the last row
        o, lse = run(k1, v, q)
        assert torch.equal(o[:, :, :3], good_o[:, :, :3])
        assert torch.equal(lse[:, :, :3], good_lse[:, :, :3])
        assert torch.isnan(o[:, :, 3]).all() and torch.isnan(lse[:, :, 3]).all()
        q1 = q.clone()
        q1[0, 1, 1, 3] = bad
        o, lse = run(k, v, q1)
        assert torch.isnan(o[0, 1, 1]).all() and torch.isnan(lse[0, 1, 1])
        o[0, 1, 1], lse[0, 1, 1] = good_o[0, 1, 1], good_lse[0, 1, 1]
        assert torch.equal(o, good_o) and torch.equal(lse, good_lse)


@pytest.mark.parametrize("power", [122, -116])
@pytest.mark.parametrize("d,Hq", [(64, 4), (128, 9), (256, 3), (64, 70), (256, 80)])
def test_queries_near_the_ends_of_the_exponents(d, Hq, power):
    """Scores of ordinary size from q near 2^126 and tiny keys, or from tiny q; O in place of q."""
    L, page = 150, 32
    k, v, q = (rand((1, h, n, d), 160 + i, BF16) for i, (h, n) in
               enumerate(((1, L), (1, L), (Hq, 1))))
    k, q = (k.float() * 2.0 ** -power).to(BF16), (q.float() * 2.0 ** power).to(BF16)
    table = widen(ints([[4, 2, 0, 1, 3]]), page)
    c = new_cache(5, 1, d, page, BF16)
    fa().cache_write(c, k.cuda(), v.cuda(), table, ints([0]))
    o, lse = fa().cache_forward(q.cuda(), c, table, ints([L]), o_dtype=torch.float32)
    qq = q.cuda()
    o2, _ = fa().cache_forward(qq, c, table, ints([L]), out=qq)
    clean()
    compare(o, lse, q, k, v, [L], None, False, None, power)
    assert o2 is qq and torch.equal(o2, o.to(BF16))


def test_a_nan_query_that_sees_nothing():
    c, table, q, k, v = attend_case(1, 2, 1, 3, [20], 64, 16, BF16, True)
    q[0, 0] = float("nan")
    o, lse = fa().cache_forward(q.cuda(), c, table.cuda(), ints([2]), causal=True)
    clean()
    assert (o[0, :, 0] == 0).all() and torch.isneginf(lse[0, :, 0]).all()
    assert torch.isnan(o[0, 0, 1:]).all() and torch.isfinite(o[0, 1]).all()


def test_zero_and_tiny_queries():
    d = 128
    c, table, q, k, v = attend_case(1, 8, 1, 1, [200], d, 64, BF16, False)
    q = torch.zeros(1, 8, 1, d, dtype=BF16)
    q[0, 1] = 1e-38
    q[0, 2] = 1e30
    q[0, 3, 0, 0], q[0, 3, 0, 1] = 1.0, 1e-6
    q[0, 4, 0, 64] = -3.0
    scale = 1.0
    o, lse = fa().cache_forward(q.cuda(), c, table.cuda(), ints([200]), scale=scale,
                                o_dtype=torch.float32)
    clean()
    keep = [0, 1, 3, 4, 5]
    compare(o[:, keep], lse[:, keep], q[:, keep], k, v, [200], None, False, scale, "tiny")
    assert torch.isfinite(o[0, 2]).all()


# ------------------------------------------------------------------ how it is called

def test_results_do_not_depend_on_timing():
    c, table, q, k, v = attend_case(3, 8, 2, 2, [5000, 17, 900], 128, 64, BF16, True)
    args = (q.cuda(), c, table.cuda(), ints([5000, 17, 900]))
    first = fa().cache_forward(*args, causal=True)
    for _ in range(5):
        again = fa().cache_forward(*args, causal=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_graph_follows_lengths_and_pages():
    """One captured step (write a token, attend) replayed as the sequences grow, then with
    other pages; two graphs with a workspace of their own each."""
    B, H, d, page, steps, pages = 2, 2, 64, 16, 20, 64  # tables for far longer sequences
    k, v = rand((B, H, steps, d), 81, BF16), rand((B, H, steps, d), 82, BF16)
    q = rand((B, 4, steps, d), 83, BF16)
    table, pool = random_table(B, pages, seed=8)
    c = new_cache(pool, H, d, page, BF16)
    kk, vv, qq = k[:, :, :1].cuda(), v[:, :, :1].cuda(), q[:, :, :1].cuda()
    tb, start, lengths = table.cuda(), ints([0, 0]), ints([1, 1])
    ws = torch.empty(fa().cache_forward_workspace_bytes(4, H, 1, d, pages * page),
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(qq), torch.empty(B, 4, 1, device="cuda")

    def step():
        fa().cache_write(c, kk, vv, tb, start)
        fa().cache_forward(qq, c, tb, lengths, causal=True, out=out, lse=lse, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = torch.cuda.CUDAGraph()
    with torch.cuda.graph(other):  # its workspace comes from the graph's own pool
        o2, lse2 = fa().cache_forward(qq, c, tb, lengths, causal=True)
    for i in range(steps):
        kk.copy_(k[:, :, i:i + 1])
        vv.copy_(v[:, :, i:i + 1])
        qq.copy_(q[:, :, i:i + 1])
        start.fill_(i)
        lengths.fill_(i + 1)
        graph.replay()
        other.replay()
        torch.cuda.synchronize()
        compare(out, lse, q[:, :, i:i + 1], k, v, [i + 1] * B, None, True, None, i)
        assert torch.equal(out, o2) and torch.equal(lse, lse2)
    tb.copy_(table.flip(0))  # the sequences change places
    graph_out = out.clone()
    other.replay()
    torch.cuda.synchronize()
    clean()
    compare(o2, lse2, q[:, :, -1:], k.flip(0), v.flip(0), [steps] * B, None, True, None, "swapped")
    assert not torch.equal(o2, graph_out)


def test_two_calls_at_once_on_two_streams():
    c, table, q, k, v = attend_case(2, 8, 2, 1, [3000, 2999], 128, 64, BF16, True)
    args = (c, table.cuda(), ints([3000, 2999]))
    q1, q2 = q.cuda(), (-q).cuda()
    want = [fa().cache_forward(x, *args, causal=True) for x in (q1, q2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(10):
        got = []
        for s, x in zip(streams, (q1, q2)):
            with torch.cuda.stream(s):
                got.append(fa().cache_forward(x, *args, causal=True))
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    clean()


def test_shared_pages():
    """Two sequences that share the pages of a common prefix."""
    d, H, page = 128, 1, 16
    k, v = rand((1, H, 32, d), 91, BF16), rand((1, H, 32, d), 92, BF16)
    k1, v1 = rand((2, H, 5, d), 93, BF16), rand((2, H, 5, d), 94, BF16)
    table = ints([[0, 1, 2], [0, 1, 3]])
    c = new_cache(4, H, d, page, BF16)
    fa().cache_write(c, k.cuda(), v.cuda(), table[:1], ints([0]))
    fa().cache_write(c, k1.cuda(), v1.cuda(), table, ints([32, 32]), ints([5, 3]))
    q = rand((2, 4, 1, d), 95, BF16)
    o, lse = fa().cache_forward(q.cuda(), c, table, ints([37, 35]), causal=True)
    clean()
    both = [torch.cat([x.expand(2, -1, -1, -1), y], 2) for x, y in ((k, k1), (v, v1))]
    compare(o, lse, q, both[0], both[1], [37, 35], None, True, None, "shared")


def test_serving_run():
    """A prompt, a chunk, then tokens one by one, against the plain implementation; and a
    causal pass of the 16-bit kernels over what was read back."""
    B, Hq, Hk, d, page = 2, 8, 2, 128, 32
    total = 170
    k, v, q = (rand((B, h, total, d), 100 + i, BF16) for i, h in enumerate((Hk, Hk, Hq)))
    table, pool = random_table(B, -(-total // page), seed=4)
    table = table.cuda()
    c = new_cache(pool, Hk, d, page, BF16)
    at = 0
    for n in (100, 61, 1, 1, 3, 1, 1, 1, 1):
        new = slice(at, at + n)
        fa().cache_write(c, k[:, :, new].cuda(), v[:, :, new].cuda(), table, ints([at] * B))
        at += n
        o, lse = fa().cache_forward(q[:, :, new].cuda(), c, table, ints([at] * B), causal=True)
        clean()
        compare(o, lse, q[:, :, new], k[:, :, :at], v[:, :, :at], [at] * B, None, True, None, at)
    assert at == total
    k2, v2 = fa().cache_read(c, table, ints([0] * B), total)
    assert torch.equal(k2.cpu(), cache_ref.read_back(k))
    rep = lambda x: x.repeat_interleave(Hq // Hk, 1).contiguous()
    o16, lse16 = fa().forward(q.cuda(), rep(k2), rep(v2), causal=True)
    oc, lsec = fa().cache_forward(q.cuda(), c, table, ints([total] * B), causal=True)
    clean()
    # the 16-bit pass rounds K, V and P to bf16: 2^-9 each of values of size about 3
    assert (o16.float() - oc.float()).abs().max() <= 3 * 3 * 2.0 ** -8
    assert (lse16 - lsec).abs().max() <= 0.1


# ------------------------------------------------------------------ refusals and bad indices

def test_binding_refusals():
    c = new_cache(4, 2, 64, 16, BF16)
    x = torch.zeros(2, 2, 3, 64, dtype=BF16, device="cuda")
    q = torch.zeros(2, 4, 3, 64, dtype=BF16, device="cuda")
    t, n = ints([[0], [1]]), ints([3, 3])
    w, f, r = fa().cache_write, fa().cache_forward, fa().cache_read
    bad = [
        lambda: w(c, x[:, :1], x[:, :1], t, n), lambda: w(c, x, x[:, :, :2], t, n),
        lambda: w(c, x[0], x[0], t, n), lambda: w(c, x.cpu(), x.cpu(), t, n),
        lambda: w(c, x, x, t.long(), n), lambda: w(c, x, x, t[:1], n),
        lambda: w(c, x, x, t[0], n), lambda: w(c, x, x, t.cpu(), n),
        lambda: w(c, x, x, t, n.long()), lambda: w(c, x, x, t, ints([1])),
        lambda: w(c, x, x, t, None), lambda: w(c, x, x, t, n, n.cpu()),
        lambda: w(c, x, x, t, ints([1, 2, 3, 4])[::2]),
        lambda: w(c, x.transpose(2, 3), x.transpose(2, 3), t, n),
        lambda: r(c, t, n, 3, k=x[:, :1]), lambda: r(c, t, None, 3),
        lambda: f(q[:, :3], c, t, n), lambda: f(q[..., :32], c, t, n), lambda: f(q[0], c, t, n),
        lambda: f(q.cpu(), c, t, n), lambda: f(q, c, t, None), lambda: f(q, c, t, n.float()),
        lambda: f(q, c, t, n, out=q[:, :2]), lambda: f(q, c, t, n, lse=torch.zeros(2, 4, 3)),
        lambda: f(q, c, t, n, workspace=torch.zeros(64, dtype=torch.uint8)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was taken")
    for call in (lambda: w(c, x.half(), x.half(), t, n), lambda: f(q.half(), c, t, n),
                 lambda: f(q, c, t, n, scale=-1.0),
                 lambda: f(q, c, ints([[0] * 100] * 2), n,  # long tables: sequences may be split
                           workspace=torch.zeros(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(fa().FAError):
            call()
    clean()


def test_empty_calls():
    c = new_cache(4, 2, 64, 16, BF16)
    t = ints([[0], [1]])
    e = torch.zeros(2, 2, 0, 64, dtype=BF16, device="cuda")
    fa().cache_write(c, e, e, t, ints([0, 0]))
    k, v = fa().cache_read(c, t, ints([0, 0]), 0)
    assert k.shape == (2, 2, 0, 64)
    q = torch.zeros(2, 4, 0, 64, dtype=BF16, device="cuda")
    o, lse = fa().cache_forward(q, c, t, ints([0, 0]))
    assert o.shape == q.shape and lse.shape == (2, 4, 0)
    clean()


def status():
    torch.cuda.synchronize()
    return fa().device_status()


def test_bad_indices_are_skipped_and_reported():
    """The kernels' own bounds checks: nothing outside the pool is touched, what is in range is
    right, and the host learns of it."""
    d, H, page = 64, 2, 16
    k, v = rand((2, H, 40, d), 111, BF16), rand((2, H, 40, d), 112, BF16)
    q = rand((2, 4, 1, d), 113, BF16)
    c = new_cache(6, H, d, page, BF16)
    good = ints([[0, 1, 2], [3, 4, 5]])
    fa().cache_write(c, k.cuda(), v.cuda(), good, ints([0, 0]))
    assert status() == 0
    before = c.data.clone()
    bad = ints([[0, 6, 2], [3, -1, 5]])
    # writes: bad pages, tokens before and behind the table
    for table, start in ((bad, [16, 16]), (good, [-40, 48]), (good, [-41, 2 ** 31 - 1])):
        fa().cache_write(c, k[:, :, :16].cuda(), v[:, :, :16].cuda(), table, ints(start))
        code = status()
        assert code & BAD_INDEX == BAD_INDEX and (code >> 16) & 0x3FFF == 9
        assert torch.equal(c.data, before)
    # reads: zeros for what is not there
    k2, _ = fa().cache_read(c, bad, ints([0, 0]), 40)
    assert (status() >> 16) & 0x3FFF == 10
    want = cache_ref.read_back(k)
    want[:, :, 16:32] = 0
    assert torch.equal(k2.cpu(), want)
    # attention: tokens of a bad page are hidden
    o, lse = fa().cache_forward(q.cuda(), c, bad, ints([40, 40]), o_dtype=torch.float32)
    assert (status() >> 16) & 0x3FFF == 11
    seen = list(range(16)) + list(range(32, 40))
    compare(o, lse, q, k[:, :, seen], v[:, :, seen], [24, 24], None, False, None, "hidden page")
    # lengths and counts are clamped
    o, lse = fa().cache_forward(q.cuda(), c, good, ints([-5, 999]), o_dtype=torch.float32)
    assert status() & BAD_INDEX == BAD_INDEX
    assert (o[0] == 0).all() and torch.isneginf(lse[0]).all()
    assert torch.isnan(o[1]).all()  # tokens 40 .. 47 were never written
    o, _ = fa().cache_forward(q.cuda(), c, good, ints([40, 40]), counts=ints([-1, 7]))
    assert status() & BAD_INDEX == BAD_INDEX
    assert (o[0] == 0).all() and (o[1] != 0).any()
    fa().cache_write(c, k.cuda(), v.cuda(), good, ints([0, 0]), ints([-3, 41]))
    assert status() & BAD_INDEX == BAD_INDEX
    assert torch.equal(c.data, before)
    assert status() == 0
    lib = binding.load_library()
    assert lib.fa_status_string(6) == b"FA_ERR_BAD_INDEX"


@pytest.mark.parametrize("d,page,Hq", [(64, 16, 80), (128, 128, 70), (96, 256, 200), (256, 48, 80),
                                       (256, 128, 90)])
def test_bad_pages_with_many_rows(d, page, Hq):
    """A page outside the pool in the middle, found cell by cell or by the tile of keys."""
    L, n_pages = 700, -(-700 // page)
    k, v, q = (rand((1, h, n, d), 120 + i, BF16) for i, (h, n) in enumerate(((1, L), (1, L), (Hq, 1))))
    c = new_cache(n_pages, 1, d, page, BF16)
    good = widen(ints([list(range(n_pages))]), page)
    fa().cache_write(c, k.cuda(), v.cuda(), good, ints([0]))
    assert status() == 0
    bad = good.clone()
    bad[0, 1] = n_pages + 7
    for lengths in (L, L - 1):
        o, lse = fa().cache_forward(q.cuda(), c, bad, ints([lengths]), o_dtype=torch.float32)
        assert status() & BAD_INDEX == BAD_INDEX
        seen = list(range(page)) + list(range(2 * page, lengths))
        compare(o, lse, q, k[:, :, seen], v[:, :, seen], [len(seen)], None, False, None, "hidden")
    bad[:] = -1
    o, lse = fa().cache_forward(q.cuda(), c, bad, ints([L]), o_dtype=torch.float32)
    assert status() & BAD_INDEX == BAD_INDEX
    assert (o == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("d", [128, 256])
def test_many_rows_from_pages_beyond_32_bit_offsets(d):
    page = 64
    pool = (1 << 32) // (64 * 5 * d // 2) + 3
    c = fa().KVCache4(pool, 1, d, page_size=page)
    table = widen(ints([[pool - 1, 3, pool - 2]]), page)
    k, v, q = (rand((1, h, 150, d), 130 + i, BF16) for i, h in enumerate((1, 1, 2)))
    fa().cache_write(c, k.cuda(), v.cuda(), table, ints([0]))
    o, lse = fa().cache_forward(q.cuda(), c, table, ints([150]), causal=True)
    clean()
    compare(o, lse, q, k, v, [150], None, True, None, "past 4 GiB, many rows")


@pytest.mark.parametrize("Hq,Nq,d", [(2, 40, 64), (3, 100, 64), (1, 100, 256)])
def test_graph_of_many_rows_follows_lengths(Hq, Nq, d):
    """A captured chunk replayed for shorter and longer sequences, down to none."""
    page, pages = 64, 40
    L = 2000
    k, v = rand((2, 1, L, d), 141, BF16), rand((2, 1, L, d), 142, BF16)
    q = rand((2, Hq, Nq, d), 143, BF16)
    table, pool = random_table(2, pages, seed=3)
    table = table.cuda()
    c = new_cache(pool, 1, d, page, BF16)
    fa().cache_write(c, k.cuda(), v.cuda(), table, ints([0, 0]))
    qq, lengths, counts = q.cuda(), ints([L, L]), ints([Nq, Nq])
    fa().cache_forward(qq, c, table, lengths, causal=True, counts=counts)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = fa().cache_forward(qq, c, table, lengths, causal=True, counts=counts)
    for ln, ct in (([L, 17], [Nq, 5]), ([0, 129], [0, Nq]), ([1999, 1000], [1, Nq])):
        lengths.copy_(torch.tensor(ln))
        counts.copy_(torch.tensor(ct))
        graph.replay()
        clean()
        compare(o, lse, q, k, v, ln, ct, True, None, (ln, ct))


@pytest.mark.parametrize("d,Nq", [(64, 1), (128, 9), (256, 1), (64, 40), (128, 100),
                                  (256, 20), (256, 40)])
def test_stalled_copies_are_reported_and_the_context_survives(d, Nq):
    lib = binding.load_library()
    c, table, q, k, v = attend_case(1, 2, 1, Nq, [500], d, 64, BF16, True, wide=True)
    try:
        assert lib.fa_debug_configure(1, 20_000_000) == 0  # no copies, 20 ms a wait
        fa().cache_forward(q.cuda(), c, table.cuda(), ints([500]), causal=True)
        code = status()
        kernel = 12 if 2 * Nq > 64 else 11
        assert code & BAD_INDEX == 0x80000000 and (code >> 16) & 0x3FFF == kernel
    finally:
        lib.fa_debug_configure(0, 0)
    o, lse = fa().cache_forward(q.cuda(), c, table.cuda(), ints([500]), causal=True)
    clean()
    compare(o, lse, q, k, v, [500], None, True, None, "after a timeout")
