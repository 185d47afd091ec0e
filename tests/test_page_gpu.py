"""The paged 8-bit cache on the GPU against its definition in 64 bits (tests/page_oracle.py)."""
import numpy as np
import pytest
import torch

from latent_space_sparse_b200 import salsc
from tests import page_oracle as po

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


class Step:
    """A random paged cache, its step and the inputs of one layer."""

    def __init__(self, lens, news=None, hq=8, hkv=2, d=128, page=16, dtype=BF16, base=10000.0,
                 window=0, scale=0.0, spare_rows=0, seed=0, max_q=None, extra_pages=2, q_gain=1.5,
                 page_gain=0.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        held = [-(-n // page) for n in lens]
        self.n_pages, self.max_pages = sum(held) + extra_pages, max(max(held), 1) + 1
        order = torch.randperm(self.n_pages, generator=g, device=DEV).tolist()
        table, at = np.full((len(lens), self.max_pages), -1, np.int32), 0
        for b, n in enumerate(held):
            table[b, :n] = order[at:at + n]
            at += n
        self.single = news is None
        news = [1] * len(lens) if news is None else news
        self.offs = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        self.rows = int(self.offs[-1]) + spare_rows
        self.lens, self.news, self.table = list(lens), list(news), table
        self.hq, self.hkv, self.d, self.page, self.dtype = hq, hkv, d, page, dtype
        self.base, self.window, self.scale = base, window, scale
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
        pool = (self.n_pages, hkv, page, d)
        self.pools = []
        for _ in range(2):
            x = rnd(*pool)
            if page_gain:  # pages of very different magnitudes
                x = x * torch.exp2((rnd(self.n_pages, hkv, 1, 1) * page_gain).round())
            a = x.abs().amax((2, 3))
            # half the scales are powers of two, half are not
            s = torch.where(rnd(*a.shape) > 0, torch.exp2((a / 448).log2().ceil()), a / 440)
            self.pools += [(x / s[:, :, None, None]).to(torch.float8_e4m3fn), s]
        self.pools = [self.pools[0], self.pools[2], self.pools[1], self.pools[3]]
        self.q = (q_gain * rnd(self.rows, hq, d)).to(dtype)
        self.K, self.V = rnd(self.rows, hkv, d).to(dtype), rnd(self.rows, hkv, d).to(dtype)
        self.t_table = torch.from_numpy(table).to(DEV)
        self.t_lens = torch.tensor(lens, dtype=torch.int32, device=DEV)
        self.t_offs = torch.from_numpy(self.offs).to(DEV)
        self.max_q = max(news) if max_q is None else max_q
        self.cache = self.new_cache()

    def new_cache(self):
        return salsc.PagedCache(self.hq, self.hkv, self.d, self.page, self.n_pages, self.t_table,
                                self.t_lens, None if self.single else self.t_offs,
                                n_tokens=self.rows, max_q=self.max_q, rope_base=self.base,
                                softmax_scale=self.scale, window=self.window, dtype=self.dtype)

    def spec(self):
        return dict(lens=self.lens, offs=self.offs.tolist(), table=self.table.tolist(),
                    base=self.base, window=self.window, scale=self.scale)


def check_attend(s, out=None, q=None, flags=0):
    q = s.q if q is None else q
    if out is None:
        out = torch.full((s.rows, s.hq, s.d), 7.0, dtype=s.dtype, device=DEV)
        s.cache.attend(q, *s.pools, out=out)
    torch.cuda.synchronize()
    assert s.cache.flags() == flags
    ref, tol = po.attend(s.spec(), q, *s.pools, s.hq, s.dtype)
    got = out.double().cpu().numpy()
    idle = np.isnan(ref).all((1, 2))
    assert (got[idle] == 7.0).all(), "rows of no sequence were written"
    err = np.abs(got - ref)[~idle]
    assert (err <= tol[~idle]).all(), f"worst {np.nanmax(err / tol[~idle])} of the tolerance"


def check_append(s, K=None, V=None, flags=0, step=None):
    K, V = s.K if K is None else K, s.V if V is None else V
    before = [p.clone() for p in s.pools]
    want = po.append(step or s.spec(), K, V, *before)
    s.cache.append(K, V, *s.pools)
    torch.cuda.synchronize()
    assert s.cache.flags() == flags
    for (vals, tol, sc), pages, scales, was in zip(want, s.pools[:2], s.pools[2:], before):
        assert np.array_equal(scales.cpu().double().numpy(), sc), "scales"
        got = po.values(pages, scales)
        same = tol == 0
        raw, old = (x.view(torch.uint8).cpu().numpy() for x in (pages, was))
        assert np.array_equal(raw[same], old[same]), "bytes of other slots changed"
        nan = np.isnan(vals) & ~same
        assert np.isnan(got[nan]).all()
        off = np.abs(got - vals)[~same & ~nan]
        assert (off <= tol[~same & ~nan]).all(), f"worst {np.max(off / tol[~same & ~nan])}"


LENS = [0, 1, 15, 16, 17, 63, 64, 127, 128, 129, 300, 513]
FORMS = [(BF16, 128, 16, 8, 2), (BF16, 128, 64, 4, 4), (BF16, 64, 32, 16, 2), (BF16, 128, 128, 8, 8),
         (BF16, 64, 128, 3, 3), (BF16, 128, 32, 16, 1), (F32, 64, 16, 6, 2), (F32, 128, 64, 5, 1),
         (F32, 128, 128, 8, 1)]


# ---- attention

@pytest.mark.parametrize("dtype,d,page,hq,hkv", FORMS)
def test_attend_single_tokens(dtype, d, page, hq, hkv):
    check_attend(Step(LENS, None, hq, hkv, d, page, dtype, seed=11))


@pytest.mark.parametrize("dtype,d,page,hq,hkv", FORMS)
def test_attend_prompts_ragged(dtype, d, page, hq, hkv):
    # whole prompts, chunks, single tokens, nothing new, more new rows than tokens (empty rows)
    news = [0, 1, 15, 3, 17, 1, 0, 130, 128, 65, 33, 200]
    check_attend(Step(LENS, news, hq, hkv, d, page, dtype, seed=12, spare_rows=3))


@pytest.mark.parametrize("news", [2, 3, 5, 7, 16, 31])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_few_new_tokens(news, dtype):
    check_attend(Step([700, 40, news], [news] * 3, 8, 2, 128, 16, dtype, seed=news))


def test_attend_single_token_with_offsets_and_empty_slots():
    check_attend(Step([5, 0, 200, 0, 33], [1, 0, 1, 1, 1], seed=3, spare_rows=2))


def test_attend_many_sequences():
    lens = [(b * 37) % 91 for b in range(600)]
    check_attend(Step(lens, None, 4, 2, 64, 16, seed=4))
    check_attend(Step(lens, [min(n, 1 + b % 3) for b, n in enumerate(lens)], 4, 2, 64, 16, seed=5))


@pytest.mark.parametrize("single", [True, False])
def test_very_many_sequences(single):
    lens = [(b * 7) % 33 for b in range(2500)]
    news = None if single else [min(n, b % 3) for b, n in enumerate(lens)]
    s = Step(lens, news, 2, 1, 64, 16, seed=6)
    check_attend(s)
    check_append(s)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_one_long_sequence(dtype):
    check_attend(Step([20011], None, 8, 2, 128, 64, dtype, seed=6))
    check_attend(Step([9001], [70], 4, 1, 128, 128, dtype, seed=6))


@pytest.mark.parametrize("lens,news,hq,hkv,d,page,window", [
    ([1700], [1700], 8, 4, 128, 64, 0), ([1300, 900, 5], [1300, 333, 1], 6, 6, 128, 16, 0),
    ([2100], [1500], 8, 4, 64, 32, 0), ([2500, 700], [1000, 700], 16, 4, 128, 128, 300)])
def test_attend_prompt_of_several_units_and_tiles_a_cta(lens, news, hq, hkv, d, page, window):
    check_attend(Step(lens, news, hq, hkv, d, page, window=window, seed=8, page_gain=1.0))


@pytest.mark.parametrize("hq,hkv,d,page", [(16, 16, 64, 16), (32, 8, 128, 32)])
def test_attend_many_units_of_one_half_between_units_of_two(hq, hkv, d, page):
    """Runs of units with at most 128 rows, more than a CTA keeps entries for, behind larger ones."""
    g = hq // hkv
    news = [200 // g if b % 40 == 0 else 5 + (b * 11) % (128 // g - 4 if b % 8 == 0 else 3) for b in range(160)]
    lens = [m + (b * 29) % 150 for b, m in enumerate(news)]
    check_attend(Step(lens, news, hq, hkv, d, page, seed=9))


@pytest.mark.parametrize("window", [1, 2, 17, 100, 128, 129, 400])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_window(window, dtype):
    check_attend(Step(LENS, None, window=window, dtype=dtype, seed=21))
    news = [0, 1, 15, 3, 17, 1, 0, 100, 128, 65, 33, 200]
    check_attend(Step(LENS, news, window=window, dtype=dtype, seed=22))


def test_attend_window_does_not_read_pages_before_it():
    s = Step([500, 300], [3, 40], window=50)
    for b, (n, m) in enumerate(zip(s.lens, s.news)):
        s.table[b, :(n - m - 49) // s.page] = -1  # pages that no query sees, given back
    s.t_table.copy_(torch.from_numpy(s.table))
    check_attend(s)


@pytest.mark.parametrize("kw", [dict(base=0.0), dict(base=500000.0), dict(scale=0.3),
                                dict(q_gain=6.0), dict(q_gain=1e-12), dict(page_gain=2.0)])
@pytest.mark.parametrize("news", [None, [100, 60, 4]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_values(kw, news, dtype):
    check_attend(Step([257, 90, 333], news, dtype=dtype, seed=31, **kw))


@pytest.mark.parametrize("news", [None, [80, 9]])
def test_attend_ignores_what_lies_behind_the_end(news):
    s = Step([133, 9], news, page=64, extra_pages=4)
    ref = s.cache.attend(s.q, *s.pools)
    raw = [p.view(torch.uint8) for p in s.pools[:2]]
    for b, n in enumerate(s.lens):
        pg = s.table[b, n // s.page]
        for r in raw:
            r[pg, :, n % s.page:] = 0x7F  # NaN codes
    used = set(s.table[s.table >= 0].tolist())
    for pg in set(range(s.n_pages)) - used:
        for r, sc in zip(raw, s.pools[2:]):
            r[pg] = 0xFF
            sc[pg] = float("nan")
    got = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    assert torch.equal(ref, got)


@pytest.mark.parametrize("news", [None, [1, 3], [40, 130]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_nan_in_the_cache_reaches_only_rows_that_see_it(news, dtype):
    s = Step([150, 170], news, dtype=dtype)
    ref = s.cache.attend(s.q, *s.pools).clone()
    t = 148  # of sequence 0: its last row sees it; earlier rows may not
    for p in s.pools[:2]:
        p.view(torch.uint8)[s.table[0, t // s.page], 1, t % s.page, 5] = 0x7F
    got = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    sees = np.zeros(s.rows, bool)
    for i in range(s.news[0]):
        sees[s.offs[0] + i] = s.lens[0] - s.news[0] + i >= t
    sees = torch.from_numpy(sees)
    g = s.hq // s.hkv
    assert torch.isnan(got[sees][:, g:2 * g, 5]).all()  # a NaN key or value is not hidden
    assert torch.equal(got[~sees], ref[~sees])
    assert torch.equal(got[:, :g], ref[:, :g])
    assert torch.equal(got[:, 2 * g:], ref[:, 2 * g:])


@pytest.mark.parametrize("news", [None, [3, 5], [150, 60], [290, 9]])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan"), 2.0 ** 119, 2.0 ** 127])
def test_attend_scale_that_is_not_finite_reaches_only_rows_that_see_it(news, dtype, which, bad):
    """A page's scale at the end of what a prompt holds: earlier rows of the same tile do not see it."""
    s = Step([300, 60], news, dtype=dtype, seed=36)
    first = 288  # sequence 0's last page
    ref = s.cache.attend(s.q, *s.pools).clone()
    s.pools[2 if which == "k" else 3][s.table[0, first // s.page], 1] = bad
    got = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    sees = torch.tensor([i < s.news[0] and s.lens[0] - s.news[0] + i >= first for i in range(s.rows)])
    g = s.hq // s.hkv
    if not np.isfinite(bad):
        assert torch.isnan(got[sees][:, g:2 * g]).all()
    assert torch.equal(got[~sees], ref[~sees])
    assert torch.equal(got[:, :g], ref[:, :g])
    assert torch.equal(got[:, 2 * g:], ref[:, 2 * g:])


@pytest.mark.parametrize("news", [None, [3, 5], [90, 40]])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_attend_query_that_is_not_finite_spoils_its_own_row_only(news, dtype, bad):
    s = Step([150, 60], news, dtype=dtype, seed=32)
    good = s.cache.attend(s.q, *s.pools)
    q = s.q.clone()
    q[1, 3, 10] = bad
    out = s.cache.attend(q, *s.pools)
    torch.cuda.synchronize()
    assert out[1, 3].isnan().all()
    out[1, 3], good[1, 3] = 0, 0
    assert torch.equal(out, good)


@pytest.mark.parametrize("news", [None, [3, 5], [200, 40]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_scales_of_any_sign_and_zero(news, dtype):
    s = Step([300, 60], news, dtype=dtype, seed=33)
    g = torch.Generator(device=DEV).manual_seed(34)
    for scales in s.pools[2:]:
        scales *= torch.randint(-1, 2, scales.shape, generator=g, device=DEV)  # -1, 0, 1
    check_attend(s)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("news", [None, [2], [260]])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attend_scores_that_jump_by_thousands(news, dtype, d):
    """Two tokens, each far above all before it: the row's result is the later one's value."""
    n, page, first, second = 700, 16, 450, 600
    s = Step([n], news, 4, 1, d, page, dtype, base=0.0, seed=35)
    s.q.fill_(1.0)
    codes = s.pools[0].view(torch.uint8)
    codes.zero_()
    s.pools[2].fill_(1.0)
    for t, scale in ((first, 1.0), (second, 3.0)):
        pg = int(s.table[0, t // page])
        codes[pg, 0, t % page] = 0x7E  # 448
        s.pools[2][pg] = scale
    out = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    assert s.cache.flags() == 0
    m = s.rows
    vals = po.values(s.pools[1], s.pools[3])
    for i in range(m):
        pos = n - m + i
        if pos < first:
            continue  # all scores are zero
        t = second if pos >= second else first
        want = vals[s.table[0, t // page], 0, t % page]
        got = out[i].double().cpu().numpy()
        # the value's mantissa (24 bits of scale, 4 of code) in f16 or fp32, then the output's rounding
        assert (np.abs(got - want) <= (2.0 ** -8 + 2.0 ** -10 if dtype == BF16 else 2.0 ** -22) * np.abs(want)).all()


def test_one_workspace_for_steps_of_every_kind():
    """Steps of different descriptors take turns with one workspace, in stream order."""
    kinds = [Step([900, 33, 1], None, 8, 2, seed=41), Step([300, 500], [300, 9], 8, 2, seed=42),
             Step([700, 40], [1, 7], 16, 1, dtype=F32, seed=43), Step([800], None, 4, 4, 64, 32, F32, seed=44),
             Step([700, 20], [5, 3], 8, 2, seed=45)]
    own = [s.cache.attend(s.q, *s.pools) for s in kinds]
    most = max((s.cache for s in kinds), key=lambda c: c.ws.numel())
    for _ in range(3):
        for s, ref in zip(kinds, own):
            s.cache._ws = most._ws
            assert torch.equal(s.cache.attend(s.q, *s.pools), ref)


def test_attend_strided_queries_of_a_fused_projection():
    s = Step([100, 37], [30, 37], hq=8, hkv=2)
    fused = torch.randn(s.rows, 12 * s.d, device=DEV, dtype=BF16)
    check_attend(s, q=fused[:, :8 * s.d].unflatten(1, (8, s.d)))
    one = Step([100], None, hq=8, hkv=2)
    fused = torch.randn(1, 12 * s.d, device=DEV, dtype=BF16)
    check_attend(one, q=fused[:, :8 * s.d].unflatten(1, (8, s.d)))


@pytest.mark.parametrize("news", [None, [40, 130]])
def test_attend_output_at_16_bytes(news):
    s = Step([300, 140], news)
    room = torch.full((s.rows * s.hq * s.d + 8,), 7.0, dtype=s.dtype, device=DEV)
    out = room[8:].view(s.rows, s.hq, s.d)
    assert out.data_ptr() % 32 == 16
    s.cache.attend(s.q, *s.pools, out=out)
    check_attend(s, out)


def test_attend_shared_prefix_pages():
    s = Step([200, 200, 170], [5, 1, 90])
    for b in (1, 2):
        s.table[b, :6] = s.table[0, :6]
    s.table[2, 7] = s.table[2, 6]  # the same page twice in one sequence
    s.t_table.copy_(torch.from_numpy(s.table))
    check_attend(s)


@pytest.mark.parametrize("news", [None, [40, 33]])
def test_attend_bad_pages_are_left_out_and_flagged(news):
    s = Step([200, 90], news)
    s.table[0, 3], s.table[0, 8], s.table[1, 0] = s.n_pages, -5, 2 ** 31 - 1
    s.t_table.copy_(torch.from_numpy(s.table))
    check_attend(s, flags=salsc.FLAG_BAD_INDEX)


@pytest.mark.parametrize("news", [None, [3, 3], [40, 33]])
def test_attend_only_bad_pages_gives_zeros(news):
    s = Step([30, 64], news)
    s.table[0] = -1
    s.t_table.copy_(torch.from_numpy(s.table))
    check_attend(s, flags=salsc.FLAG_BAD_INDEX)


def test_lengths_and_offsets_out_of_bounds_are_cut_and_flagged():
    for news in (None, [2, 2], [40, 40]):
        s = Step([60, 60], news)
        for lens in ([-3, 60], [s.max_pages * s.page + 1, 60]):
            s.t_lens.copy_(torch.tensor(lens))
            s.cache.append(s.K, s.V, *s.pools)
            out = s.cache.attend(s.q, *s.pools)
            torch.cuda.synchronize()
            assert s.cache.flags() & salsc.FLAG_BAD_INDEX
            assert out.shape[0] == s.rows
    s = Step([60, 60], [40, 40], max_q=40)
    for offs in ([0, 90, 80], [-4, 40, 81], [0, 45, 50]):
        s.t_offs.copy_(torch.tensor(offs))
        s.cache.append(s.K, s.V, *s.pools)
        s.cache.attend(s.q, *s.pools)
        torch.cuda.synchronize()
        assert s.cache.flags() & salsc.FLAG_BAD_INDEX


@pytest.mark.parametrize("news", [None, [70]])
def test_pool_of_more_than_2_31_bytes(news):
    """Pages at the far end of pools of 2^32 bytes and more."""
    n_pages, hkv, page, d, n = (1 << 20) + 9, 4, 16, 64, 150
    table = torch.arange(n_pages - 1, n_pages - 11, -1, dtype=torch.int32, device=DEV)[None]
    pools = [torch.empty(n_pages, hkv, page, d, dtype=torch.uint8, device=DEV)
             .view(torch.float8_e4m3fn) for _ in range(2)]
    pools += [torch.ones(n_pages, hkv, device=DEV) for _ in range(2)]
    rows = 1 if news is None else news[0]
    K, V = (torch.randn(n, hkv, d, device=DEV, dtype=BF16) for _ in range(2))
    q = torch.randn(rows, 8, d, device=DEV, dtype=BF16)
    lens = torch.tensor([n], dtype=torch.int32, device=DEV)
    offs = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    cache = salsc.PagedCache(8, hkv, d, page, n_pages, table, lens, offs, n_tokens=n, max_q=n)
    cache.append(K, V, *pools)
    offs = None if news is None else torch.tensor([0, rows], dtype=torch.int32, device=DEV)
    cache = salsc.PagedCache(8, hkv, d, page, n_pages, table, lens, offs, n_tokens=rows, max_q=rows)
    out = cache.attend(q, *pools)
    torch.cuda.synchronize()
    assert cache.flags() == 0
    small = [p[-10:].contiguous() for p in pools]
    step = dict(lens=[n], offs=[0, rows], table=[list(range(9, -1, -1))], base=1e4, window=0)
    ref, tol = po.attend(step, q, *small, 8, BF16)
    assert (np.abs(out.double().cpu().numpy() - ref) <= tol).all()
    full = dict(step, offs=[0, n])
    fresh = [torch.zeros_like(small[0]), torch.zeros_like(small[1]), small[2], small[3]]
    for (vals, t, sc), pages, scales in zip(po.append(full, K, V, *fresh), small[:2], small[2:]):
        assert np.array_equal(scales.cpu().double().numpy(), sc)
        got = po.values(pages, scales)
        assert (np.abs(got - vals) <= t)[t > 0].all()


# ---- append

@pytest.mark.parametrize("dtype,d,page,hq,hkv", FORMS)
def test_append_single_tokens(dtype, d, page, hq, hkv):
    check_append(Step(LENS, None, hq, hkv, d, page, dtype, seed=41))


@pytest.mark.parametrize("dtype,d,page,hq,hkv", FORMS)
def test_append_prompts_ragged(dtype, d, page, hq, hkv):
    news = [0, 1, 15, 3, 20, 1, 0, 127, 100, 65, 33, 513]
    check_append(Step(LENS, news, hq, hkv, d, page, dtype, seed=42, spare_rows=5))


def test_append_many_sequences():
    lens = [(b * 37) % 91 for b in range(600)]
    check_append(Step(lens, None, 4, 2, 64, 16, seed=4))
    check_append(Step(lens, [min(n, 1 + b % 3) for b, n in enumerate(lens)], 4, 2, 64, 16, seed=5))


@pytest.mark.parametrize("base", [0.0, 500000.0])
def test_append_rotation(base):
    check_append(Step([131072, 40], [30, 40], base=base, page=128))


def test_append_grows_a_page_scale_and_recodes():
    for page in (16, 64, 128):
        s = Step([page - 2, page - 2, page - 2], [2, 1, 5], page=page)
        for gain in (64.0, 1e-3, 3.0e4):
            check_append(s, s.K * gain, s.V * gain)


def test_append_twice_is_the_same():
    s = Step([40, 77], [5, 30])
    s.cache.append(s.K * 9, s.V * 9, *s.pools)
    once = [p.clone() for p in s.pools]
    s.cache.append(s.K * 9, s.V * 9, *s.pools)
    for a, b in zip(once, s.pools):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_zeros_infinities_nan_and_extremes(dtype):
    s = Step([40, 70], [17, 70], dtype=dtype)
    K, V = s.K.clone(), s.V.clone()
    K[3:12], V[3:12] = 0.0, 0.0
    K[20, 0], V[20, 0] = 0.0, 0.0
    V[25, 1, 7], V[26, 0, 9], V[27, 0, 1] = float("inf"), float("-inf"), float("nan")
    K[30, 1, 3] = float("nan")  # its pair becomes NaN
    V[40, 0], V[60, 1] = 3e38, 1e-38
    K[45, 0, 5] = 2e38
    check_append(s, K, V)


def test_append_strided_rows_of_a_fused_projection():
    s = Step([100, 37], [30, 37], hq=8, hkv=2)
    fused = torch.randn(s.rows, 12 * s.d, device=DEV, dtype=BF16).unflatten(1, (12, s.d))
    check_append(s, fused[:, 8:10], fused[:, 10:])


def test_append_bad_pages_are_skipped_and_flagged():
    s = Step([100, 40], [50, 3])
    good = s.spec()
    s.table[0, 4] = s.n_pages + 7
    s.t_table.copy_(torch.from_numpy(s.table))
    before = [p.clone() for p in s.pools]
    s.cache.append(s.K, s.V, *s.pools)
    torch.cuda.synchronize()
    assert s.cache.flags() == salsc.FLAG_BAD_INDEX
    skipped = good["table"][0][4]
    for a, b in zip(before, s.pools):
        assert torch.equal(a[skipped].view(torch.uint8), b[skipped].view(torch.uint8))
    want = po.append(good, s.K, s.V, *before)
    rest = [p for p in range(s.n_pages) if p != skipped]
    for (vals, tol, sc), pages, scales in zip(want, s.pools[:2], s.pools[2:]):
        assert np.array_equal(scales.cpu().double().numpy()[rest], sc[rest])
        off = np.abs(po.values(pages, scales) - vals)[rest]
        written = tol[rest] > 0
        assert (off[written] <= tol[rest][written]).all()


def test_append_more_rows_than_tokens_skips_the_first():
    check_append(Step([5, 0, 20], [9, 4, 20]))


# ---- as they are used

def drive(s, layers, steps, graph, stream):
    """A prompt, then single tokens, over several layers' caches; returns the outputs."""
    outs = []
    g = torch.Generator(device=DEV).manual_seed(9)
    pools = [salsc.alloc_pages(s.n_pages, s.hkv, s.page, s.d) for _ in range(layers)]
    rnd = lambda n, h: torch.randn(n, h, s.d, generator=g, device=DEV).to(s.dtype)  # noqa: E731
    with torch.cuda.stream(stream):
        prompt = s.new_cache()
        for p in pools:
            prompt.append(rnd(s.rows, s.hkv), rnd(s.rows, s.hkv), *p)
            outs.append(prompt.attend(rnd(s.rows, s.hq), *p))
        B = len(s.lens)
        lens = s.t_lens.clone()
        table = s.t_table.clone()
        one = salsc.PagedCache(s.hq, s.hkv, s.d, s.page, s.n_pages, table, lens, dtype=s.dtype)
        K, V, q = (rnd(B * layers, h).view(layers, B, h, s.d) for h in (s.hkv, s.hkv, s.hq))
        out = torch.zeros_like(q)

        def step():
            for i, p in enumerate(pools):
                one.append(K[i], V[i], *p)
                one.attend(q[i], *p, out=out[i])

        if graph:
            before = [[x.clone() for x in p] for p in pools]
            lens.add_(1)
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg, stream=stream):
                step()
            lens.sub_(1)
            for p, old in zip(pools, before):
                for x, o in zip(p, old):
                    x.copy_(o)
        for _ in range(steps):
            lens.add_(1)
            for x, h in ((K, s.hkv), (V, s.hkv), (q, s.hq)):
                x.copy_(rnd(B * layers, h).view(x.shape))
            cg.replay() if graph else step()
            outs.append(out.clone())
        torch.cuda.synchronize()
        assert one.flags() == 0 and prompt.flags() == 0
    return outs, pools


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_prompt_then_tokens_eager_graph_and_other_stream_agree(dtype):
    s = Step([45 + 16, 130 + 16, 3 + 16], [45, 130, 3], dtype=dtype)  # room for what comes
    s.lens = [45, 130, 3]
    s.t_lens.copy_(torch.tensor(s.lens))
    first, pools = drive(s, 2, 9, False, torch.cuda.current_stream())
    again, _ = drive(s, 2, 9, True, torch.cuda.Stream())
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    # the last step's output against the definition over the final caches
    last = dict(lens=[n + 9 for n in s.lens], offs=[0, 1, 2, 3], table=s.table.tolist(), base=1e4,
                window=0)
    g = torch.Generator(device=DEV).manual_seed(9)
    for _ in range(2):
        for h in (s.hkv, s.hkv, s.hq):
            torch.randn(s.rows, h, s.d, generator=g, device=DEV)
    for _ in range(10):
        K, V, q = (torch.randn(6, h, s.d, generator=g, device=DEV).to(dtype).view(2, 3, h, s.d)
                   for h in (s.hkv, s.hkv, s.hq))
    for i in range(2):
        ref, tol = po.attend(last, q[i], *pools[i], s.hq, dtype)
        assert (np.abs(first[-1][i].double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_mixed_step_in_a_graph_serves_changing_lengths(dtype):
    s = Step([700, 90, 400, 16], [300, 1, 40, 2], dtype=dtype, max_q=512, spare_rows=200, seed=51)
    out = torch.zeros(s.rows, s.hq, s.d, dtype=dtype, device=DEV)
    g = torch.cuda.CUDAGraph()
    s.cache.attend(s.q, *s.pools, out=out)
    with torch.cuda.graph(g):
        s.cache.append(s.K, s.V, *s.pools)
        s.cache.attend(s.q, *s.pools, out=out)
    for lens, news in (([700, 90, 400, 16], [300, 1, 40, 2]), ([650, 96, 1, 0], [500, 6, 1, 0]),
                       ([33, 33, 33, 16], [1, 1, 1, 1])):
        s.lens, s.news, s.offs = lens, news, np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        s.t_lens.copy_(torch.tensor(lens))
        s.t_offs.copy_(torch.from_numpy(s.offs))
        out.fill_(7.0)
        g.replay()
        check_attend(s, out)


def test_two_caches_on_two_streams_at_once():
    a, b = Step([3000, 2000], None, seed=1), Step([900, 1200], [300, 250], seed=2)
    ra, rb = (s.cache.attend(s.q, *s.pools).clone() for s in (a, b))
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = [], []
    for _ in range(20):
        oa.append(a.cache.attend(a.q, *a.pools, stream=sa))
        ob.append(b.cache.attend(b.q, *b.pools, stream=sb))
    torch.cuda.synchronize()
    assert all(torch.equal(x, ra) for x in oa) and all(torch.equal(x, rb) for x in ob)


def test_attend_is_the_same_every_time():
    s = Step([5000, 131, 77], [1, 131, 50], seed=8)
    ref = s.cache.attend(s.q, *s.pools)
    for _ in range(5):
        assert torch.equal(s.cache.attend(s.q, *s.pools), ref)


def test_binding_checks_its_tensors():
    s = Step([20], None)
    for bad in (s.q.float(), s.q[:, :4], s.q.cpu(), s.q.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            s.cache.attend(bad, *s.pools)
    with pytest.raises(ValueError):
        s.cache.attend(s.q, *s.pools, out=torch.empty(1, 8, 256, device=DEV, dtype=BF16)[..., ::2])
    for i in range(4):
        pools = list(s.pools)
        pools[i] = pools[i][:-1]
        with pytest.raises(ValueError):
            s.cache.append(s.K, s.V, *pools)
    with pytest.raises(ValueError):
        s.cache.append(s.K, s.V.float(), *s.pools)


def test_empty_step():
    s = Step([0, 0], [0, 0])
    s.cache.append(s.K, s.V, *s.pools)
    assert s.cache.attend(s.q, *s.pools).shape == (0, 8, 128)
    assert s.cache.flags() == 0
