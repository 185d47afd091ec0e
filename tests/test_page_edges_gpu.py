"""The paged 8-bit cache at the edges of what its calls take, against its definition in 64 bits
(tests/page_oracle.py)."""
import numpy as np
import pytest
import torch

from latent_space_sparse_b200 import salsc, synth, workloads
from tests import page_oracle as po
from tests.test_page_gpu import BF16, DEV, F32, Step, check_append, check_attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news", [None, [100, 3], [4, 3]])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("code", [0x38, 0xB8])  # 1, -1
@pytest.mark.parametrize("pos,base", [(0, 0.0), (1, 0.0), (0, 10000.0), (1, 10000.0)])
def test_attend_infinite_query_whose_scores_are_all_minus_infinity(dtype, news, bad, code, pos, base):
    """(Away from position 0 the rotation spreads an infinity over its pair without making a NaN.)"""
    n0 = news[0] if news else pos + 1
    s = Step([n0, 60], news, dtype=dtype, base=base, seed=37)
    row = pos if news else 0
    s.pools[0].view(torch.uint8)[s.table[0, 0], 1, :pos + 1, 10::64] = code  # a pair of all that the row sees
    good = s.cache.attend(s.q, *s.pools)
    q = s.q.clone()
    q[row, 5, 10] = bad  # head 5 reads KV head 1
    out = s.cache.attend(q, *s.pools)
    torch.cuda.synchronize()
    assert out[row, 5].isnan().all()
    out[row, 5], good[row, 5] = 0, 0
    assert torch.equal(out, good)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news", [None, [3, 5]])
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("old", [-1.0, -0.25, 0.0, -2.0 ** 20, -3.0e-7, 2.0 ** 127, float("inf"),
                                 float("-inf"), float("nan")])
def test_append_behind_a_page_scale_of_any_kind_keeps_the_earlier_tokens(dtype, news, page, old):
    """Earlier tokens keep what they stand for (code * scale); where that is not finite, NaN."""
    lens = [page + 9, page + 12]
    s = Step(lens, news, page=page, dtype=dtype, seed=38)
    for b in range(2):
        for scales in s.pools[2:]:
            scales[s.table[b, 1]] = old
    before = [p.clone() for p in s.pools]
    s.cache.append(s.K, s.V, *s.pools)
    torch.cuda.synchronize()
    assert s.cache.flags() == 0
    for x, pages, scales, p0, s0 in zip((s.K, s.V), s.pools[:2], s.pools[2:], before[:2], before[2:]):
        x = x.double().cpu().numpy()
        got, was = po.values(pages, scales), po.values(p0, s0)
        for b, n in enumerate(lens):
            m = s.news[b]
            pg, lo = s.table[b, 1], n - m - page
            size = np.abs(x[s.offs[b]:s.offs[b] + m])
            if pages is s.pools[0]:
                size = size[..., :s.d // 2] + size[..., s.d // 2:]
            for u in range(s.hkv):
                need = po.scale_for(size[:, u].max())
                want = max(need, abs(old)) if np.isfinite(old) else need
                assert float(scales[pg, u]) == want
                a, e = got[pg, u, :lo], was[pg, u, :lo]
                if np.isfinite(old):
                    assert (np.abs(a - e) <= po.half_step(e, want)).all()
                else:
                    assert np.isnan(a).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news", [None, [3, 2], [150, 90]])
@pytest.mark.parametrize("zero,rest", [(-100, 30), (-100, 50), (-100, -60), (-60, 40), (-99, 0), (119, 119),
                                       (119, 20), (120, 120), (127, 127), (127, 30), (-100, -99), (-100, -80),
                                       (-100, 120), (-100, 127), (-101, -101), (-99, -99), (-101, -98)])
def test_attend_value_scales_far_apart(dtype, news, zero, rest):
    """Pages of zeros beside pages of any magnitude (the append gives them a scale of 2^-100), and
    value scales far from one."""
    s = Step([200, 150], news, dtype=dtype, seed=39)
    g = torch.Generator(device=DEV).manual_seed(3)
    small = torch.rand(s.n_pages, generator=g, device=DEV) < 0.5
    s.pools[3] = torch.where(small[:, None], 2.0 ** zero, 2.0 ** rest).float().expand(-1, s.hkv).contiguous()
    if zero == -100:
        s.pools[1].view(torch.uint8)[small] = 0
    elif zero == -101:  # the append's scale for zeros and the smallest values
        s.pools[3].clamp_(min=2.0 ** -100)
    if max(zero, rest) > 100:  # values that stay finite in bf16
        top = 200.0 if max(zero, rest) < 127 else 1.5
        s.pools[1] = s.pools[1].float().clamp(-top, top).to(torch.float8_e4m3fn)
    check_attend(s)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news", [None, [3], [100]])
@pytest.mark.parametrize("times", [8.5, 10.5, 13.5, 20.3, 42.5])
def test_attend_small_weights_beside_a_large_one(dtype, news, times):
    """A first token that takes all the weight and has no value (a sink), and others at
    times * 2^-24 of it, whose values are the result. (One tile: one maximum for all.)"""
    n, d, far = 120, 128, 24 - np.log2(times)
    s = Step([n], news, 4, 1, d, 64, dtype, base=0.0, seed=48)
    s.q.fill_(1.0)
    codes, values = (p.view(torch.uint8) for p in s.pools[:2])
    codes.zero_()
    first = int(s.table[0, 0])
    codes[first, 0, 0] = 0x38  # 1: its score is sqrt(d) times its page's key scale
    values[first, 0, 0] = 0
    s.pools[2].fill_(1.0)
    s.pools[2][first] = far * np.log(2.0) / np.sqrt(d)
    s.pools[3].fill_(1.0)
    values &= 0x7F  # positive: no cancellation
    values.clamp_(max=0x40)  # at most 2
    out = s.cache.attend(s.q, *s.pools).double().cpu().numpy()
    step = dict(s.spec(), base=0.0)
    ref, _ = po.attend(step, s.q, *s.pools, 4, dtype)
    # a weight: its own floor, and the score's roundings (three factors and a sum at `far` log2
    # units, each by half a step of 2^-23 relative); fp32 sums of 128 terms, twice; the
    # output's rounding
    floor, own = (2.0 ** -27, 2.0 ** -8) if dtype == BF16 else (2.0 ** -42, 2.0 ** -24)
    rel = floor * 2.0 ** far + 4 * far * 2.0 ** -24 + 2 * 128 * 2.0 ** -24 + own
    if dtype == BF16:
        rel += 2.0 ** -11
    assert (np.abs(out - ref) <= rel * np.abs(ref)).all(), np.max(np.abs(out - ref) / np.abs(ref)) / rel


@pytest.mark.parametrize("news", [None, [3, 2], [40, 30]])
def test_attend_queries_at_the_end_of_fp32(news):
    s = Step([70, 50], news, dtype=F32, base=0.0, seed=40)
    s.q *= 3.3e38 / s.q.abs().amax()
    s.pools[2] *= 2.0 ** -123
    check_attend(s)


def test_constructor_is_ordered_before_calls_on_other_streams():
    s = Step([3000, 2000], None, seed=45)
    ref = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        junk = [torch.full((s.cache.ws.numel() + 256,), 255, dtype=torch.uint8, device=DEV) for _ in range(3)]
        torch.cuda.synchronize()
        del junk  # the next workspace's memory
        torch.cuda._sleep(20_000_000)
        cache = s.new_cache()
        out = cache.attend(s.q, *s.pools, stream=side)
        torch.cuda.synchronize()
        assert cache.flags() == 0
        assert torch.equal(out, ref)


def test_output_allocated_for_a_stream_belongs_to_it():
    s = Step([300, 200], None, seed=46)
    ref = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(3):
        old = torch.empty_like(ref)
        torch.cuda._sleep(20_000_000)
        old.fill_(1.0)  # not done yet when its memory is free again
        del old
        out = s.cache.attend(s.q, *s.pools, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.parametrize("news", [None, [30, 1, 9]])
def test_every_new_token_counts_where_max_q_is_not_given(news):
    s = Step([40, 33, 9], news, seed=49)
    s.cache = salsc.PagedCache(s.hq, s.hkv, s.d, s.page, s.n_pages, s.t_table, s.t_lens,
                               None if s.single else s.t_offs, n_tokens=s.rows)
    check_attend(s)
    check_append(s)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("hq,hkv,news", [(8, 2, None), (32, 32, None), (8, 8, [60, 1, 1, 9, 1, 33] * 5),
                                         (32, 8, [60, 1, 1, 9, 1, 33] * 5)])
def test_attend_right_behind_an_append_reads_what_it_wrote(dtype, hq, hkv, news):
    """Scales of a page's heads lie side by side and are written by different CTAs; each step lets
    the last pages' scales grow."""
    lens = [(37 * b) % 200 + 61 for b in range(30)]
    s = Step(lens, news, hq, hkv, 64, 128, dtype, seed=47)
    pools = [p.clone() for p in s.pools]
    for i in range(12):
        K, V = s.K * 1.9 ** i, s.V * 1.9 ** i
        s.cache.append(K, V, *pools)
        got = s.cache.attend(s.q, *pools)
        torch.cuda.synchronize()
        assert torch.equal(got, s.cache.attend(s.q, *pools)), i


def _cut(s, lens, offs):
    """The sequences as the entry points cut them: (tokens, first row, new rows, sequence)."""
    cap, seqs = s.max_pages * s.page, []
    for b, n in enumerate(lens):
        o0 = min(max(offs[b], 0), s.rows)
        o1 = min(max(offs[b + 1], o0), s.rows)
        seqs.append((min(max(n, 0), cap), o0, min(o1 - o0, s.max_q), b))
    return seqs


@pytest.mark.parametrize("news,max_q,lens,offs", [
    (None, 1, [-3, 60], [0, 1, 2]), (None, 1, [81, 60], [0, 1, 2]), (None, 1, [2 ** 31 - 1, 60], [0, 1, 2]),
    ([2, 2], 2, [-3, 60], [0, 2, 4]), ([2, 2], 2, [81, 60], [0, 2, 4]),
    ([40, 40], 40, [-2 ** 31, 60], [0, 40, 80]), ([40, 40], 40, [60, 81], [0, 40, 80]),
    ([40, 40], 50, [60, 60], [0, 90, 80]), ([40, 40], 40, [60, 60], [-4, 30, 60]),
    ([40, 40], 80, [60, 60], [0, 40, 81]), ([40, 40], 80, [60, 60], [-2 ** 31, 40, 2 ** 31 - 1]),
    ([40, 40], 40, [60, 60], [0, 45, 50]), ([40, 40], 40, [60, 60], [0, 10, 80]),
    ([2, 2], 2, [60, 60], [0, 3, 4]), ([40, 40], 80, [60, 60], [0, 80, 40])])
@pytest.mark.parametrize("what", ["append", "attend"])
def test_each_length_and_offset_out_of_bounds_is_cut_and_flagged(news, max_q, lens, offs, what):
    s = Step([60, 60], news, max_q=max_q, seed=44)
    assert s.max_pages * s.page == 80
    # the last page of each exists, so that nothing but the length or offset is wrong
    s.table[:, 4] = sorted(set(range(s.n_pages)) - set(s.table[s.table >= 0].tolist()))
    s.t_table.copy_(torch.from_numpy(s.table))
    s.t_lens.copy_(torch.tensor(lens))
    s.t_offs.copy_(torch.tensor(offs))
    before = [p.clone() for p in s.pools]
    out = torch.full((s.rows, s.hq, s.d), 7.0, dtype=s.dtype, device=DEV)
    if what == "append":
        s.cache.append(s.K, s.V, *s.pools)
    else:
        s.cache.attend(s.q, *s.pools, out=out)
    torch.cuda.synchronize()
    assert s.cache.flags() == salsc.FLAG_BAD_INDEX
    if what == "attend":
        want, off = np.full(out.shape, 7.0), np.zeros(out.shape)
        for n, row, m, b in _cut(s, lens, offs):
            one = dict(s.spec(), lens=[n], offs=[row, row + m], table=[s.table[b].tolist()])
            ref, tol = po.attend(one, s.q, *s.pools, s.hq, s.dtype)
            want[row:row + m], off[row:row + m] = ref[row:row + m], tol[row:row + m]
        assert (np.abs(out.double().cpu().numpy() - want) <= off).all()
        return
    scales = [x.cpu().double().numpy() for x in before[2:]]
    vals = [po.values(p, x) for p, x in zip(before[:2], before[2:])]
    tols = [np.zeros(v.shape) for v in vals]
    for n, row, m, b in _cut(s, lens, offs):
        one = dict(s.spec(), lens=[n], offs=[row, row + m], table=[s.table[b].tolist()])
        for i, (v, t, sc) in enumerate(po.append(one, s.K, s.V, *before)):
            for pg in set(np.nonzero(t)[0].tolist()):
                vals[i][pg], tols[i][pg], scales[i][pg] = v[pg], t[pg], sc[pg]
    for v, t, sc, pages, got, was in zip(vals, tols, scales, s.pools[:2], s.pools[2:], before):
        assert np.array_equal(got.cpu().double().numpy(), sc)
        assert (np.abs(po.values(pages, got) - v)[t > 0] <= t[t > 0]).all()
        raw, old = (x.view(torch.uint8).cpu().numpy() for x in (pages, was))
        assert np.array_equal(raw[t == 0], old[t == 0])


@pytest.mark.parametrize("news", [None, [200, 1, 9]])
@pytest.mark.parametrize("graph", [False, True])
def test_compressed_and_full_layers_take_turns_on_one_stream(news, graph):
    """A model's layers: latent decode steps and paged steps one after another, launched early on
    each other's heels, give what each gives alone."""
    w = workloads.Workload(name="layers", batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, rank=128,
                           top_k=256, seq_lens=(1500, 700), dtype="bf16", rope_base=10000.0,
                           low_rank=16, seed=62)
    x = {k: v.to(DEV) for k, v in synth.decode_inputs(w).items() if k in ("q", "Kc", "Vc", "Pk", "Pv")}
    dec = salsc.Decoder(w.batch, w.n_q_heads, w.n_kv_heads, w.head_dim, w.rank, w.top_k, w.seq_lens,
                        rope_base=w.rope_base, dtype=BF16, device=DEV)
    s = Step([1200, 900, 309], news, seed=50)
    s.cache.append(s.K, s.V, *s.pools)
    torch.cuda.synchronize()
    latent = dec.step(**x)
    torch.cuda.synchronize()
    full = s.cache.attend(s.q, *s.pools)
    torch.cuda.synchronize()
    a, b = ([torch.zeros_like(t) for _ in range(6)] for t in (latent, full))

    def layers():
        for i in range(6):
            s.cache.append(s.K, s.V, *s.pools)  # the same tokens again
            s.cache.attend(s.q, *s.pools, out=b[i])
            dec.step(**x, out=a[i])

    if graph:
        layers()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layers()
        for t in a + b:
            t.zero_()
        g.replay()
        g.replay()
    else:
        layers()
    torch.cuda.synchronize()
    assert dec.flags() == 0 and s.cache.flags() == 0
    assert all(torch.equal(t, latent) for t in a)
    assert all(torch.equal(t, full) for t in b)
