"""The serving operators on the GPU where they can go wrong beside the sizes and masks of test_serving.py, against the
references and tolerances of serving_ref.py."""
import pytest
import torch

from tests import serving_ref as R
from tests.test_serving import DEV, Case, _rsq, gen, i32

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------------------------- int64 block tables

def i64(v):
    return torch.tensor(v, dtype=torch.int64, device=DEV)


@pytest.mark.parametrize("size", [16, 128])
def test_plan_of_an_int64_table(size):
    rsq = _rsq()
    ctx, new, width, T = [0, 5, size, 3 * size - 1, 0], [1, 2 * size, 0, 1, 3], 5, 2 * size + 9
    table = [[700 + 10 * b + j for j in range(width)] for b in range(len(ctx))]
    ids = list(range(40, 60))
    want = R.plan(ctx, new, table, ids, 2, T, size)
    t = i64(table)
    cu, seq, pos, slots, cur = rsq.kv8_plan(i32(ctx), i32(new), t, i32(ids), i32([2]), T, size)
    assert rsq.device_status() == 0 and t.dtype == torch.int64
    assert (t.tolist(), cu.tolist(), seq.tolist(), pos.tolist(), slots.tolist(), cur.item()) == want
    # the free list and the table's columns end
    for n_free, columns in ((1, 5), (20, 2)):
        cut = [r[:columns] for r in table]
        want = R.plan(ctx, new, cut, ids[:n_free], 0, T, size)
        t = i64(cut)
        got = rsq.kv8_plan(i32(ctx), i32(new), t, i32(ids[:n_free]), i32([0]), T, size)
        assert rsq.device_status() == 16
        assert (t.tolist(), *(x.tolist() for x in got[:4]), got[4].item()) == want


def test_plan_of_ids_that_no_cache_has():
    """Ids from 2^31 - 1 on become slots that the append reports and skips; negative ones become slot -1."""
    rsq = _rsq()
    t = i64([[1 << 31], [(1 << 32) + 1], [1 << 62], [-1 << 40], [1]])
    _, _, _, slots, _ = rsq.kv8_plan(i32([3] * 5), i32([1] * 5), t, i32([9]), i32([0]), 5, 16)
    assert slots.tolist() == [((1 << 31) - 1) * 16 + 3] * 3 + [-1, 19]
    kc = torch.zeros((2, 1, 16, 16), dtype=torch.int8, device=DEV)
    ks = torch.zeros((2, 1), device=DEV)
    vc, vs = kc.clone(), ks.clone()
    x = torch.ones((5, 16), device=DEV)
    rsq.kv8_append(x, x, slots, kc, ks, vc, vs)
    assert rsq.device_status() == 8
    assert kc.count_nonzero().item() == 16 and (kc[1, 0, 3] == 127).all()


INT64_CASES = [([(100, 1), (300, 3), (0, 0)], 16, 4, 2, 64, torch.bfloat16), ([(5000, 1), (20, 2)], 64, 8, 2, 128, torch.bfloat16),
               ([(90, 4), (7, 1)], 32, 5, 1, 128, torch.float32), ([(60, 3)], 16, 2, 1, 256, torch.float32),
               ([(1500, 300), (0, 800), (45, 4)], 16, 4, 2, 128, torch.bfloat16),
               ([(1500, 300), (0, 800), (45, 4)], 128, 4, 2, 64, torch.bfloat16)]


@pytest.mark.parametrize("lens,size,H,kv,dh,dtype", INT64_CASES)
def test_attention_of_an_int64_table(lens, size, H, kv, dh, dtype):
    """The same bits as with an int32 table; ids that would be valid by their low 32 bits are not."""
    rsq = _rsq()
    c = Case(lens, size, H, kv, dh, dtype, 17)
    args = [x.to(DEV) for x in (c.q, c.kc, c.ks, c.vc, c.vs)]
    lists = i32(c.seq), i32(c.cu)
    assert torch.equal(rsq.kv8_attention(*args, i64(c.table), *lists), rsq.kv8_attention(*args, i32(c.table), *lists))
    assert rsq.device_status() == 0
    for b, n in enumerate(c.seq):
        if n:
            c.table[b][n // size // 2] = -1
    want = rsq.kv8_attention(*args, i32(c.table), *lists)
    assert rsq.device_status() == 8
    for bad in ((1 << 32) + 1, 1 << 40, -1 << 33, c.n_blocks):
        table = [[bad if j == -1 else j for j in r] for r in c.table]
        assert torch.equal(rsq.kv8_attention(*args, i64(table), *lists), want)
        assert rsq.device_status() == 8


def test_tables_of_other_types_are_refused():
    rsq = _rsq()
    c = Case([(30, 1)], 16, 2, 1, 64, torch.bfloat16, 3)
    args = [x.to(DEV) for x in (c.q, c.kc, c.ks, c.vc, c.vs)]
    before = rsq.launch_count()
    for dtype in (torch.int16, torch.float32, torch.uint8):
        t = i32(c.table).to(dtype)
        with pytest.raises(TypeError):
            rsq.kv8_attention(*args, t, i32(c.seq), i32(c.cu))
        with pytest.raises(TypeError):
            rsq.kv8_plan(i32([0]), i32([1]), t, i32([1]), i32([0]), 1, 16)
    with pytest.raises(ValueError):
        rsq.kv8_attention(*args, i64(c.table).repeat(1, 2)[:, ::2], i32(c.seq), i32(c.cu))
    assert rsq.launch_count() == before


# ---------------------------------------------------------------------------------------------- values that are no numbers

# 256 rows (new tokens x heads of a group) and 2^19 pairs of a row and a token make a request long
LONG = [(0, 800), (45, 4), (1500, 300)]


@pytest.mark.parametrize("size", [16, 32, 64, 128])
@pytest.mark.parametrize("dh", [64, 128])
def test_attention_long_chunks_with_bad_values_in_front(dh, size):
    """A block whose value scale is NaN or infinite reaches every row that sees it, also where it is the first that a row
    sees, or all that it sees, or the rest of its 128 keys weighs nothing."""
    for bad in (float("nan"), float("inf")):
        c = Case(LONG, size, 4, 2, dh, torch.bfloat16, 21)
        first = [c.table[0][0], c.table[2][0]]
        c.vs[first] = bad
        c.check("first block")
        c.vs[[c.table[b][j] for b in (0, 2) for j in range(1, 128 // size)]] = 0.0
        c.check("first block, no weight on the rest of the tile")
        c.vs[[c.table[b][j] for b in (0, 2) for j in range(128 // size)]] = bad
        c.check("the first 128 tokens")
        c = Case(LONG, size, 4, 2, dh, torch.bfloat16, 22)
        c.vs[[j for j in c.table[2] if j >= 0], 0] = bad
        c.vs[[j for j in c.table[0] if j >= 0], 1] = 0.0
        c.vs[c.table[0][300 // size], 1] = bad
        c.check("a head of nothing else, one among zeros")


@pytest.mark.parametrize("dh,size", [(64, 128), (128, 16), (128, 128)])
def test_attention_long_chunks_with_bad_values_in_every_piece(dh, size):
    """The keys of a few tiles of rows are spread over the GPU in pieces: wherever the poisoned 128 tokens lie, all rows see
    them."""
    c = Case([(20000, 130)], size, 4, 1, dh, torch.bfloat16, 23)
    q, kc, ks, vc = (x.to(DEV) for x in (c.q, c.kc, c.ks, c.vc))
    table, seq, cu = i32(c.table), i32(c.seq), i32(c.cu)
    clean = c.vs.to(DEV)
    outs = []
    for tile in range(0, 156, 5):
        vs = clean.clone()
        vs[c.table[0][tile * 128 // size:(tile + 1) * 128 // size]] = float("nan")
        outs.append(_rsq().kv8_attention(q, kc, ks, vc, vs, table, seq, cu).isnan().all())
    assert torch.stack(outs).all(), [5 * i for i, o in enumerate(outs) if not o]
    assert not _rsq().kv8_attention(q, kc, ks, vc, clean, table, seq, cu).isnan().any()


@pytest.mark.parametrize("size", [16, 128])
@pytest.mark.parametrize("dh", [64, 128])
def test_attention_long_chunks_with_bad_blocks_anywhere(dh, size):
    """Poisoned, foreign and missing blocks at the beginning, inside and at the end of requests of many pairs."""
    for where in (0.0, 0.1, 0.5, 0.9):
        c = Case(LONG, size, 4, 2, dh, torch.bfloat16, 26)
        at = [int(where * s) // size for s in c.seq]
        c.ks[c.table[0][at[0]], 0] = float("nan")
        c.ks[c.table[2][at[2]], 1] = float("inf")
        c.vs[c.table[2][at[2]], 0] = float("inf")
        c.check(f"poisoned at {where}")
        c = Case(LONG, size, 4, 2, dh, torch.bfloat16, 27)
        c.table[0][at[0]] = 1 << 30
        c.table[1][at[1]] = c.n_blocks
        c.table[2][at[2]] = -1
        c.check(f"foreign at {where}", want_status=8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
def test_attention_bad_values_that_weigh_nothing(dh, dtype):
    """A NaN value scale counts also where the block's probabilities are below the smallest number."""
    for size in (16, 64):
        lens = [(90, 1), (300, 60), (17, 3)] + ([(0, 800)] if dtype == torch.bfloat16 and dh >= 64 else [])
        c = Case(lens, size, 4, 2, dh, dtype, 24, sharp=400.0)
        for r in c.table:
            c.vs[r[0]] = float("nan")
        c.check(f"size={size}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [16, 64, 128])
def test_attention_of_queries_that_are_no_numbers(dh, dtype):
    """An infinity in a query makes every score infinite or NaN and the row NaN, also where all of them are -infinity, and no
    other row.  (The others keep to the references' tolerance, not to the bits without it: 32 rows of a long chunk take the
    products of probabilities and value scales in one way or the other together, each within that tolerance.)"""
    for size in (16, 64):
        lens = [(0, 1), (40, 1), (0, 20), (300, 60)] + ([(0, 800)] if dtype == torch.bfloat16 and dh >= 64 else [])
        c = Case(lens, size, 4, 2, dh, dtype, 25)
        c.kc[..., 5] = -c.kc[..., 5].abs().clamp(min=1)     # no zero code meets the infinity
        head = torch.arange(4) * dh + 5
        rows = list(range(0, len(c.q), 3))
        c.q[rows[0::3], head[1]] = float("inf")
        c.q[rows[1::3], head[1]] = float("-inf")
        c.q[rows[2::3], head[1]] = float("nan")
        assert c.run().reshape(-1, 4, dh)[rows, 1].isnan().all()
        c.check(f"size={size}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [16, 32, 256])
def test_attention_several_tokens_of_other_head_sizes(dh, dtype):
    for i, (H, kv) in enumerate([(1, 1), (8, 2), (5, 1), (32, 2)]):
        size = (16, 32, 64, 128)[i]
        lens = [(0, 2), (40, 3), (0, 0), (size - 1, 2), (100, 17), (size, 5), (0, 33), (3, 140)]
        Case(lens, size, H, kv, dh, dtype, 28 + i, pad=2, strided=i % 2 == 1).check(f"H={H} kv={kv}")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [64, 128])
def test_attention_of_a_query_element_far_above_the_rest(dh, dtype):
    """The largest element of a row is 2^32 times the rest and meets only codes of 0.  Each of the others is off by up to
    2^-39 of it, so a score by E = |sm_scale| 2^-39 max |q| sum |k| and a probability by exp(E) - 1 of itself; the output by
    that twice (numerator and denominator) times A."""
    for size in (16, 64):
        lens = [(300, 1), (40, 70)] + ([(0, 800)] if dtype == torch.bfloat16 else [])
        c = Case(lens, size, 4, 2, dh, dtype, 31)
        c.kc[..., 7] = 0
        c.q.reshape(-1, 4, dh)[..., 7] = 2.0 ** 32
        got = c.run().cpu().double().reshape(-1, 4, dh)
        want, big, S = R.attention(c.q, c.kc, c.ks, c.vc, c.vs, c.table, c.seq, c.cu, c.sm)
        keys = (c.kc.double().abs().sum(-1) * c.ks.double()[..., None]).amax()
        E = c.sm * 2.0 ** -39 * 2.0 ** 32 * keys
        assert E < 0.5
        tol = R.attention_tol(want, big, S, max(c.seq), dh, dtype) + 2 * torch.expm1(E) * big
        assert ((got - want).abs() <= tol).all(), f"size={size}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("dh", [32, 64, 128])
def test_attention_without_a_scale_of_scores(dh, dtype):
    """sm_scale 0: the mean of what a row sees."""
    for size in (16, 64):
        c = Case([(0, 1), (77, 3), (0, 800)], size, 2, 2, dh, dtype, 32)
        c.sm = 0.0
        c.check(f"size={size}")


# ---------------------------------------------------------------------------------------------- 4-bit weights

@pytest.mark.parametrize("group", [32, 64, 96, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matvec_keeps_infinities(dtype, group):
    """An infinity in x gives an infinity of the formula's sign, NaN where it meets a code of 0 or another sign; NaN gives NaN,
    whichever bits of its payload are set."""
    rsq = _rsq()
    g = gen(group)
    for T in (1, 3, 6, 8, 9, 20, 24, 25, 33, 48, 64, 70):
        N, K = 150, 4 * group
        x = torch.randn((T, K), generator=g).to(dtype)
        x[0, 17] = float("inf")
        x[T // 2, K - 3] = float("-inf")
        if T > 4:
            x[T - 1, 40], x[T - 1, 2] = float("inf"), float("-inf")
            x[1, 33] = float("nan")
            if dtype == torch.float32:
                x.view(torch.int32)[2, 9] = 0x7F800001      # a NaN whose upper half is that of an infinity
        codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
        scales = torch.exp(torch.randn((N, K // group), generator=g)) * 0.01
        want, big = R.matvec(x, codes, scales)
        got = rsq.w4_matvec(x.to(DEV), codes.to(DEV), scales.to(DEV), out_dtype=torch.float32).cpu().double()
        assert torch.equal(got.isnan(), want.isnan()), f"T={T}: NaN in other places"
        inf = want.isinf()
        assert inf.any() and torch.equal(got.isinf(), inf) and torch.equal(got[inf], want[inf]), f"T={T}"
        fine = want.isfinite()
        tol = R.matvec_tol(want, big, K, torch.float32)
        assert ((got - want).abs()[fine] <= tol[fine]).all(), f"T={T}"


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matvec_of_the_largest_x_there_may_be(dtype):
    """|x| < 2^118: the products of a group with the codes stay finite before they meet its scale."""
    rsq = _rsq()
    for group in (32, 128):
        for T in (2, 7, 30, 66):
            x = torch.full((T, 256), 2.0 ** 118).to(dtype)
            x[:, ::2] *= 1 - torch.finfo(dtype).eps / 2      # the largest below it
            x[:, 1::2] = x[:, ::2]
            x[1] = -x[1]
            codes = torch.full((20, 128), 0x88, dtype=torch.uint8)      # -8
            scales = torch.full((20, 256 // group), 2.0 ** -30)
            want, big = R.matvec(x, codes, scales)
            got = rsq.w4_matvec(x.to(DEV), codes.to(DEV), scales.to(DEV), out_dtype=torch.float32).cpu().double()
            assert ((got - want).abs() <= R.matvec_tol(want, big, 256, torch.float32)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 96])
def test_matvec_is_exact_on_whole_numbers_for_any_rows(group, dtype):
    """Whole x and scales of powers of two: every sum is exact, in both kernels and their variants."""
    rsq = _rsq()
    g = gen(group)
    for T in (1, 6, 9, 17, 24, 30, 33, 48, 64, 70):
        K = group * 9
        x = torch.randint(-8, 9, (T, K), generator=g).to(dtype)
        codes = torch.randint(0, 256, (140, K // 2), generator=g, dtype=torch.uint8)
        scales = 2.0 ** torch.randint(-2, 3, (140, 9), generator=g).float()
        want, _ = R.matvec(x, codes, scales)
        got = rsq.w4_matvec(x.to(DEV), codes.to(DEV), scales.to(DEV), out_dtype=torch.float32)
        assert torch.equal(got.cpu().double(), want), f"T={T}"
