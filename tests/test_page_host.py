"""The paged 8-bit cache without a GPU: refusals of the entry points (each returns before any CUDA
work is enqueued) and pins of the oracle."""
import ctypes

import numpy as np
import pytest
import torch

from latent_space_sparse_b200 import salsc
from tests import page_oracle as po

OK, INVALID, UNSUPPORTED, WORKSPACE = (salsc.SALSC_OK, salsc.SALSC_ERR_INVALID_ARG,
                                       salsc.SALSC_ERR_UNSUPPORTED, salsc.SALSC_ERR_WORKSPACE)


def desc(**kw):
    a = dict(batch=3, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=50,
             max_pages=10, n_tokens=7, max_q=4, page_table_dev=1 << 20, seq_lens_dev=1 << 21,
             q_offsets_dev=1 << 22, rope_base=10000.0, softmax_scale=0.0, window=0,
             dtype=salsc.SALSC_BF16)
    a.update(kw)
    return salsc.PageDesc(**a)


def size(d):
    return salsc.load().salsc_page_workspace_size(ctypes.byref(d))


def append(d, k=1 << 23, ks=0, v=1 << 24, vs=0, pools=(1 << 25, 1 << 26, 1 << 27, 1 << 28),
           ws=1 << 30, nb=1 << 32):
    return salsc.load().salsc_page_append(ctypes.byref(d), k, ks, v, vs, *pools, ws, nb, None)


def attend(d, q=1 << 23, qs=0, pools=(1 << 25, 1 << 26, 1 << 27, 1 << 28), out=1 << 24,
           ws=1 << 30, nb=1 << 32):
    return salsc.load().salsc_page_attend(ctypes.byref(d), q, qs, *pools, out, ws, nb, None)


BAD = [(dict(batch=0), INVALID), (dict(n_q_heads=7), INVALID), (dict(n_kv_heads=0), INVALID),
       (dict(head_dim=0), INVALID), (dict(page_size=0), INVALID), (dict(n_pages=0), INVALID),
       (dict(max_pages=0), INVALID), (dict(n_tokens=-1), INVALID), (dict(max_q=-1), INVALID),
       (dict(window=-1), INVALID), (dict(dtype=2), INVALID), (dict(rope_base=1.0), INVALID),
       (dict(rope_base=float("inf")), INVALID), (dict(rope_base=float("nan")), INVALID),
       (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID),
       (dict(page_table_dev=None), INVALID), (dict(seq_lens_dev=None), INVALID),
       (dict(q_offsets_dev=None, n_tokens=2), INVALID),  # fewer rows than sequences
       (dict(head_dim=96), UNSUPPORTED), (dict(page_size=24), UNSUPPORTED),
       (dict(page_size=256), UNSUPPORTED), (dict(n_q_heads=34), UNSUPPORTED),
       (dict(n_q_heads=257, n_kv_heads=257), UNSUPPORTED),
       (dict(n_pages=1 << 27), UNSUPPORTED),      # n_pages * 2 * 16 = 2^32 rows
       (dict(max_pages=1 << 27), UNSUPPORTED)]    # positions past 2^31


@pytest.mark.parametrize("kw,status", BAD)
def test_bad_descriptors(kw, status):
    d = desc(**kw)
    assert size(d) == 0
    assert append(d) == status
    assert attend(d) == status
    assert salsc.load().salsc_page_prepare(ctypes.byref(d), 1 << 30, 1 << 32, None) == status


@pytest.mark.parametrize("kw", [{}, dict(rope_base=0.0), dict(n_q_heads=32), dict(max_q=0),
                                dict(q_offsets_dev=None), dict(dtype=salsc.SALSC_F32, head_dim=64),
                                dict(page_size=128), dict(n_q_heads=256, n_kv_heads=256)])
def test_good_descriptors_have_a_workspace(kw):
    assert size(desc(**kw)) >= 256


def test_null_descriptor():
    lib = salsc.load()
    assert lib.salsc_page_workspace_size(None) == 0
    assert lib.salsc_page_prepare(None, 1 << 30, 1 << 32, None) == INVALID


def test_append_pointers_strides_workspace():
    d = desc()
    assert append(d, k=None) == INVALID
    assert append(d, v=None) == INVALID
    assert append(d, k=(1 << 23) + 8) == INVALID
    assert append(d, v=(1 << 24) + 2) == INVALID
    for i in range(4):
        for bad in (None, (1 << 25) + 2):
            pools = [1 << 25, 1 << 26, 1 << 27, 1 << 28]
            pools[i] = bad
            assert append(d, pools=pools) == INVALID
    assert append(d, ks=255) == INVALID   # shorter than a row
    assert append(d, vs=260) == INVALID   # not a multiple of 8
    assert append(d, ks=-256) == INVALID
    assert append(d, ws=None) == WORKSPACE
    assert append(d, ws=(1 << 30) + 128) == WORKSPACE
    assert append(d, nb=size(d) - 1) == WORKSPACE


def test_attend_pointers_strides_workspace():
    d = desc()
    assert attend(d, q=None) == INVALID
    assert attend(d, out=None) == INVALID
    assert attend(d, q=(1 << 23) + 8) == INVALID
    assert attend(d, out=(1 << 24) + 4) == INVALID
    for i in range(4):
        pools = [1 << 25, 1 << 26, 1 << 27, 1 << 28]
        pools[i] = None
        assert attend(d, pools=pools) == INVALID
    assert attend(d, qs=1016) == INVALID
    assert attend(d, qs=1028) == INVALID
    assert attend(d, ws=None) == WORKSPACE
    assert attend(d, ws=(1 << 30) + 16) == WORKSPACE
    assert attend(d, nb=size(d) - 1) == WORKSPACE


def test_attend_refuses_an_output_over_its_queries():
    """Pieces of a row's work read its queries when others may have written its output."""
    d = desc()  # rows of 1024 bf16: 2048 bytes, 7 of them
    q = 1 << 23
    for out in (q, q + 16, q + 7 * 2048 - 16, q - 7 * 2048 + 16):
        assert attend(d, q=q, out=out) == INVALID
    for out in (q, q + 6 * 2560 + 2048 - 16):
        assert attend(d, q=q, qs=1280, out=out) == INVALID


def test_nothing_to_do_is_ok_and_launches_nothing():
    for kw in (dict(n_tokens=0), dict(max_q=0)):
        d = desc(**kw)
        assert append(d, k=None if kw.get("n_tokens") == 0 else 1 << 23) == OK
        assert attend(d) == OK


def test_nothing_to_do_without_offsets():
    d = desc(q_offsets_dev=None, max_q=0)
    assert append(d) == OK
    assert attend(d) == OK


def test_binding_refuses_cpu_tensors():
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        salsc.PagedCache(8, 2, 128, 16, 9, t, torch.ones(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        salsc.PagedCache(8, 2, 128, 16, 9, t.long(), torch.ones(2, dtype=torch.int32))


def bare_cache(dtype=torch.bfloat16):
    """A PagedCache's checks of its tensors, without a GPU."""
    c = object.__new__(salsc.PagedCache)
    c.dtype, c.device, c._dev = dtype, torch.device("cpu"), -1
    return c


def test_binding_refuses_rows_that_overlap():
    """A row stride of 0 means contiguous to the entry points: rows expanded from one would be read
    behind its end."""
    c, shape = bare_cache(), (5, 4, 128)
    one = torch.zeros(1, 4, 128, dtype=torch.bfloat16)
    for bad in (one.expand(shape), torch.zeros(5 * 512, dtype=torch.bfloat16).as_strided(shape, (504, 128, 1))):
        with pytest.raises(ValueError):
            c._rows("q", bad, shape)
    with pytest.raises(ValueError):  # expanded over the heads
        c._rows("q", torch.zeros(5, 1, 128, dtype=torch.bfloat16).expand(shape), shape)
    assert c._rows("q", one, (1, 4, 128)) == 0
    assert c._rows("q", torch.zeros(shape, dtype=torch.bfloat16), shape) == 0
    fused = torch.zeros(5, 12, 128, dtype=torch.bfloat16)
    assert c._rows("K_new", fused[:, 4:8], shape) == 12 * 128
    assert c._rows("K_new", fused[:, 4:5], (5, 1, 128)) == 12 * 128
    # the stride of a single head does not matter
    assert c._rows("K_new", fused.as_strided((5, 1, 128), (1536, 7, 1)), (5, 1, 128)) == 12 * 128


def test_binding_refuses_a_stream_of_another_device():
    class Stream:
        device_index, cuda_stream = 1, 0

    c = bare_cache()
    c._dev = 0
    with pytest.raises(ValueError):
        c._call(None, "salsc_page_append", Stream())


# ---- oracle pins

def test_oracle_code_table_is_e4m3():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(codes, po.E4M3, equal_nan=True)


def test_oracle_scale():
    for a, s in ((448.0, 1.0), (448.0001, 2.0), (224.0, 0.5), (1.75, 2.0 ** -8), (0.0, 2.0 ** -100)):
        assert po.scale_for(a) == s


def test_oracle_rotation_is_relative_and_keeps_the_norm():
    r = np.random.default_rng(3)
    x, y = r.standard_normal(64), r.standard_normal(64)
    assert np.isclose(np.linalg.norm(po.rotate(x, 1234, 1e4)), np.linalg.norm(x))
    assert np.isclose(po.rotate(x, 17, 1e4) @ po.rotate(y, 12, 1e4), po.rotate(x, 5, 1e4) @ y)
    a = 3.0 * 1e4 ** -(1 / 32)  # pair 1 of 32 at position 3, by hand
    z = po.rotate(x, 3, 1e4)
    assert np.isclose(z[1], x[1] * np.cos(a) - x[33] * np.sin(a))
    assert np.isclose(z[33], x[33] * np.cos(a) + x[1] * np.sin(a))


def test_oracle_attention_is_the_library_formula():
    r = torch.Generator().manual_seed(5)
    U, G, T, d, n = 2, 3, 16, 64, 37
    k = torch.randn(3, U, T, d, generator=r).to(torch.float8_e4m3fn)
    v = torch.randn(3, U, T, d, generator=r).to(torch.float8_e4m3fn)
    ks, vs = torch.rand(3, U, generator=r) + 0.5, torch.rand(3, U, generator=r) + 0.5
    q = torch.randn(4, U * G, d, generator=r)
    step = dict(lens=[n], offs=[0, 4], table=[[2, 0, 1]], base=0.0, window=0)
    out, _ = po.attend(step, q, k, v, ks, vs, U * G, torch.float32)
    full = [torch.cat([(x[p].double() * s[p].double()[:, None, None]) for p in (2, 0, 1)], 1)[:, :n]
            for x, s in ((k, ks), (v, vs))]
    kk, vv = (x.repeat_interleave(G, 0) for x in full)
    mask = torch.arange(n)[None] <= torch.arange(n - 4, n)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), kk, vv,
                                                           attn_mask=mask)
    assert np.allclose(out, ref.transpose(0, 1).numpy(), atol=1e-12)
