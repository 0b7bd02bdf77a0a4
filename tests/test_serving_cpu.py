"""Argument checks of the table, K/V cache, attention and norm entry points (no GPU): a refused call
returns its code and message before it touches a device."""

import ctypes

import pytest

P = ctypes.c_void_p
FAKE = P(0x1000)


def cache(**kw):
    from dsa_sparse_attention_fp8_gb300.binding import KvCache
    d = dict(k=0x1000, v=0x2000, k_scale=None, v_scale=None, k_page_stride=64 * 8 * 128, k_token_stride=8 * 128,
             k_head_stride=128, v_page_stride=64 * 8 * 128, v_token_stride=8 * 128, v_head_stride=128,
             k_scale_page_stride=512, k_scale_head_stride=64, v_scale_page_stride=512, v_scale_head_stride=64,
             num_pages=16, num_kv_heads=8, head_dim=128, type=0)
    d.update(kw)
    return KvCache(**d)


def attention(lib, c, type=0, T=4, Hq=64, R=1, q=FAKE, stride=64 * 128, scale=0.1, window=0, sinks=0, ws=FAKE,
              ws_bytes=1 << 40, max_blocks=4, meta=FAKE, out=FAKE):
    return lib.dsa_paged_attention(q, stride, 128, type, T, Hq, ctypes.byref(c) if c else None, meta, meta, R, meta,
                                   max_blocks, scale, window, sinks, out, 64 * 128, 128, None, ws, ws_bytes, None, None)


def write(lib, c, type=0, T=4, k=FAKE, stride=1024, slots=FAKE):
    return lib.dsa_kv_write(k, stride, 128, FAKE, 1024, 128, type, T, slots, ctypes.byref(c) if c else None, None, None)


BAD_CACHES = [
    (dict(num_kv_heads=0), -1), (dict(head_dim=24), -2), (dict(head_dim=144), -2), (dict(head_dim=0), -2),
    (dict(num_pages=0), -1), (dict(num_pages=1 << 40), -1), (dict(k=None), -1), (dict(v=0x2008), -1),
    (dict(k_token_stride=1025), -1), (dict(v_page_stride=-1024), -1), (dict(type=2), -2), (dict(type=1), -2),
    (dict(type=3), -1),                                                  # E4M3 without scales
    (dict(type=3, k_scale=0x1000, v_scale=0x1004), -1),                  # misaligned scales
    (dict(type=3, k_scale=0x1000, v_scale=0x1000, k_scale_head_stride=65), -1),
]


@pytest.mark.parametrize("change,code", BAD_CACHES)
def test_bad_caches_are_refused(lib, change, code):
    c = cache(**change)
    assert write(lib, c) == code and lib.dsa_last_error()
    assert attention(lib, c) == code and lib.dsa_last_error()


def test_a_dimension_of_one_may_have_any_stride(lib):
    """Nothing is ever a stride away (a transposed [pages, 64, 1] scale counts as contiguous with a head stride of 1)."""
    one = dict(num_kv_heads=1, num_pages=1, type=3, k_scale=0x1000, v_scale=0x1000, k_page_stride=7, v_page_stride=-3,
               k_head_stride=1, v_head_stride=5, k_scale_page_stride=3, v_scale_page_stride=-1, k_scale_head_stride=1,
               v_scale_head_stride=2)
    c = cache(**one)
    assert write(lib, c, T=0) == 0 and attention(lib, c, T=0) == 0
    for name, size in (("num_kv_heads", 8), ("num_pages", 16)):
        assert write(lib, cache(**{**one, name: size}), T=0) == -1
    assert write(lib, cache(type=3, k_scale=0x1000, v_scale=0x1000, k_scale_page_stride=-4), T=0) == -1


def test_attention_refusals(lib):
    c = cache()
    assert attention(lib, None) == -1
    assert attention(lib, c, T=-1) == -1
    assert attention(lib, c, R=0) == -1
    assert attention(lib, c, type=2) == -2                                # FP32 rows
    assert attention(lib, c, Hq=12) == -2                                 # not a multiple
    assert attention(lib, c, Hq=0) == -2
    assert attention(lib, cache(num_kv_heads=1), Hq=129) == -2            # too many query heads to a key head
    assert attention(lib, cache(type=3, k_scale=0x1000, v_scale=0x1000), type=1) == -2   # E4M3 with FP16 rows
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attention(lib, c, scale=scale) == -1
    assert attention(lib, c, window=-1) == -1 and attention(lib, c, sinks=-1) == -1
    assert attention(lib, c, max_blocks=0) == -1
    assert attention(lib, c, q=None) == -1 and attention(lib, c, out=None) == -1 and attention(lib, c, meta=None) == -1
    assert attention(lib, c, q=P(0x1008)) == -1 and attention(lib, c, stride=8193) == -1
    assert attention(lib, c, ws=None) == -1 and attention(lib, c, ws=P(0x1010)) == -1
    assert attention(lib, c, ws_bytes=16) == -3
    assert attention(lib, c, T=0, q=None) == 0 and lib.dsa_last_launch_count() == 0


def test_write_refusals(lib):
    c = cache()
    assert write(lib, None) == -1
    assert write(lib, c, T=-1) == -1
    assert write(lib, c, type=2) == -2
    assert write(lib, c, k=None) == -1 and write(lib, c, slots=None) == -1
    assert write(lib, c, k=P(0x1002)) == -1 and write(lib, c, stride=1023) == -1
    assert write(lib, c, T=0, k=None) == 0 and lib.dsa_last_launch_count() == 0


def test_table_refusals(lib):
    def build(q=FAKE, R=4, free=FAKE, num_free=8, max_blocks=4, T=4, out=FAKE):
        return lib.dsa_block_tables_build(q, FAKE, R, free, num_free, FAKE, max_blocks, T, out, FAKE, FAKE, FAKE, None,
                                          None)
    assert build(T=-1) == -1 and build(R=0) == -1 and build(max_blocks=0) == -1 and build(num_free=-1) == -1
    assert build(R=16385) == -2 and b"16384" in lib.dsa_last_error()
    assert build(q=None) == -1 and build(free=None) == -1 and build(out=None) == -1


def test_norm_refusals(lib):
    def norm(x=FAKE, stride=256, weight=FAKE, type=0, T=4, N=256, eps=1e-6, out=FAKE, codes=FAKE, scales=FAKE, res=None):
        return lib.dsa_add_rms_norm(x, stride, res, 255, weight, type, T, N, eps, None, 0, out, 256, codes, scales, None)
    assert norm(T=-1) == -1 and norm(N=0) == -1 and norm(N=32769, stride=40000) == -2 and norm(type=3) == -2
    assert norm(eps=-1.0) == -1 and norm(eps=float("nan")) == -1
    assert norm(out=None, codes=None, scales=None) == -1
    assert norm(scales=None) == -1 and norm(codes=None) == -1
    assert norm(stride=255) == -1 and norm(res=FAKE) == -1
    assert norm(x=None) == -1 and norm(weight=None) == -1
    assert norm(T=0, x=None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import torch

    from dsa_sparse_attention_fp8_gb300 import binding as B
    x = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.kv_write(x, x, torch.zeros(2, dtype=torch.int64), x, x)
    with pytest.raises(TypeError):
        B.kv_write(x.double(), x, None, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        B.add_rms_norm(x[0], None, x[0, 0], 1e-6, out=x[0])
    with pytest.raises(ValueError, match="scales go"):
        B._kv_cache(x, x, x.float(), x.float(), x, 4, 64, 0)
    with pytest.raises(ValueError, match="needs k_scale"):
        B._kv_cache(x.view(torch.uint8), x.view(torch.uint8), None, None, x, 4, 128, 0)
    with pytest.raises(ValueError, match="shape"):
        B._kv_cache(x, x, None, None, x, 4, 64, 0)          # 4 tokens to a page
    y = torch.zeros(2, 64, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B._kv_cache(y, y, None, None, x, 4, 64, 0)
    with pytest.raises(TypeError, match="k_cache must be"):
        B._kv_cache(y.half(), y, None, None, x, 4, 64, 0)


def test_the_cache_description_matches_the_c_struct(lib):
    """The packed bytes that the binding hands over are the fields of dsa_kv_cache."""
    from dsa_sparse_attention_fp8_gb300 import binding as B
    values = list(range(1, 19))
    got = B.KvCache.from_buffer_copy(B._KV_CACHE.pack(*values).ljust(ctypes.sizeof(B.KvCache), b"\0"))
    assert [getattr(got, n) for n, _ in B.KvCache._fields_] == values
    assert B._KV_CACHE.size <= ctypes.sizeof(B.KvCache) <= B._KV_CACHE.size + 4
