"""Argument checks of the products, the router and the experts' sum (no GPU): a refused call returns its code and message
before it touches a device."""

import ctypes

import pytest

P = ctypes.c_void_p
FAKE = P(0x1000)


def fp8(lib, x=FAKE, stride=256, scales=FAKE, T=4, w=FAKE, w_stride=256, w_scales=FAKE, N=256, K=256, gated=0, out=FAKE,
        out_stride=256, out_type=0, codes=None, out_scales=None):
    return lib.dsa_fp8_matmul(x, stride, scales, T, w, w_stride, w_scales, N, K, gated, out, out_stride, out_type, codes,
                              out_scales, None, None)


def grouped(lib, x=FAKE, stride=256, scales=FAKE, type=3, S=4, rows=None, M=4, w=FAKE, w_row=256, w_group=65536, w_scales=FAKE,
            N=256, K=256, starts=FAKE, E=4, gated=0, out=FAKE, out_stride=256, out_type=0, codes=None, out_scales=None):
    return lib.dsa_grouped_matmul(x, stride, scales, type, S, rows, M, w, w_row, w_group, w_scales, N, K, starts, E, gated, out,
                                  out_stride, out_type, codes, out_scales, None, None)


SHARED = [
    (dict(N=0), -1), (dict(K=0), -1), (dict(N=257, gated=1), -1), (dict(N=192, gated=1), -2), (dict(out=None), -1),
    (dict(codes=FAKE, out_scales=FAKE), -1), (dict(out=None, codes=FAKE, gated=1), -1), (dict(codes=FAKE), -1),
    (dict(out=None, codes=FAKE, out_scales=FAKE), -2), (dict(out_type=3), -2), (dict(out_stride=255), -1),
    (dict(stride=257), -1), (dict(stride=-256), -1), (dict(stride=0), -1), (dict(x=None), -1), (dict(x=P(0x1008)), -1),
    (dict(scales=None), -1), (dict(w_scales=None), -1), (dict(w=None), -1), (dict(w=P(0x1001)), -1), (dict(out=P(0x1001)), -1),
]


@pytest.mark.parametrize("change,code", SHARED)
def test_products_refuse(lib, change, code):
    assert fp8(lib, **change) == code and lib.dsa_last_error()
    assert grouped(lib, **change) == code and lib.dsa_last_error()


def test_dense_product_refusals(lib):
    assert fp8(lib, T=-1) == -1 and fp8(lib, w_stride=250) == -1 and fp8(lib, w_stride=0) == -1
    assert fp8(lib, T=(1 << 30) + 1) == -2 and fp8(lib, N=(1 << 28) + 1) == -2 and fp8(lib, K=(1 << 28) + 1) == -2
    assert fp8(lib, T=0, x=None, w=None) == 0 and lib.dsa_last_launch_count() == 0


def test_grouped_product_refusals(lib):
    assert grouped(lib, type=2) == -2 and grouped(lib, type=7) == -2
    assert grouped(lib, E=0) == -1 and grouped(lib, E=1025) == -2
    assert grouped(lib, M=5) == -1 and b"x_rows" in lib.dsa_last_error()       # no rows, but another number of them
    assert grouped(lib, S=0, rows=FAKE) == -1 and grouped(lib, starts=None) == -1
    assert grouped(lib, w_row=0) == -1 and grouped(lib, w_group=0) == -1 and grouped(lib, w_group=8) == -1
    assert grouped(lib, type=0, w_row=260) == -1 and grouped(lib, type=0, stride=260) == -1   # multiples of 8 elements
    assert grouped(lib, S=1 << 20, stride=1 << 20, rows=FAKE) == -2 and b"64 GB" in lib.dsa_last_error()
    assert grouped(lib, M=0, S=0, x=None) == 0 and grouped(lib, M=0, rows=FAKE, starts=None) == 0


def route(lib, logits=FAKE, stride=256, type=2, T=4, E=256, k=8, scoring=0, groups=8, top_groups=4, scale=1.0, ids=FAKE,
          starts=FAKE):
    return lib.dsa_route_experts(logits, stride, type, None, T, E, k, scoring, groups, top_groups, 1, scale, None, ids, FAKE,
                                 starts, FAKE, FAKE, None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), -1), (dict(E=0), -1), (dict(E=513), -2), (dict(type=3), -2), (dict(k=0), -1), (dict(k=17), -2),
    (dict(scoring=2), -1), (dict(groups=0), -1), (dict(groups=7), -1), (dict(groups=64, top_groups=64), -2),
    (dict(top_groups=0), -1), (dict(top_groups=9), -1), (dict(groups=128, E=512), -2), (dict(groups=32, top_groups=1, k=9), -1),
    (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(T=1 << 27, k=9), -2), (dict(stride=255), -1),
    (dict(logits=None), -1), (dict(ids=None), -1), (dict(starts=None), -1),
])
def test_router_refuses(lib, change, code):
    assert route(lib, **change) == code and lib.dsa_last_error()


def combine(lib, y=FAKE, stride=64, type=0, M=8, places=FAKE, T=4, k=2, N=64, add=None, add_stride=64, out=FAKE, out_stride=64):
    return lib.dsa_combine_experts(y, stride, type, M, places, FAKE, T, k, N, add, add_stride, out, out_stride, None, None)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), -1), (dict(M=-1), -1), (dict(N=0), -1), (dict(k=0), -1), (dict(k=17), -2), (dict(type=3), -2),
    (dict(N=(1 << 28) + 1, stride=1 << 29, out_stride=1 << 29), -2), (dict(stride=63), -1), (dict(out_stride=63), -1), (dict(add=FAKE, add_stride=63), -1), (dict(y=None), -1),
    (dict(places=None), -1), (dict(out=None), -1), (dict(y=P(0x1001)), -1), (dict(out=P(0x1001)), -1),
])
def test_combine_refuses(lib, change, code):
    assert combine(lib, **change) == code and lib.dsa_last_error()


def test_combine_of_nothing(lib):
    assert combine(lib, T=0, places=None) == 0 and lib.dsa_last_launch_count() == 0


class On:
    """Makes host tensors that say they lie on cuda:0, or another device."""

    def __new__(cls, t, device=0):
        import torch

        class Fake(torch.Tensor):
            is_cuda = True

            def get_device(self):
                return device
        return t.as_subclass(Fake)


def test_the_binding_checks_its_tensors(monkeypatch):
    import torch

    from dsa_sparse_attention_fp8_gb300 import binding as B
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "load", lambda: pytest.fail("the call went on"))
    u8, f32, bf, i32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32

    def t(*shape, dtype=f32, device=0):
        return On(torch.zeros(*shape, dtype=dtype), device)
    x, xs, w, ws = t(4, 256, dtype=u8), t(4, 2), t(128, 256, dtype=u8), t(1, 2)
    starts, rows = t(4, dtype=i32), t(6, dtype=i32)
    w3, ws3 = t(3, 128, 256, dtype=u8), t(3, 1, 2)
    out = t(4, 128, dtype=bf)
    host = torch.zeros(4, 256, dtype=u8)
    for error, match, call in [
        (ValueError, "CUDA", lambda: B.fp8_matmul(host, xs, w, ws)),
        (ValueError, "cuda:1.*cuda:0", lambda: B.fp8_matmul(t(4, 256, dtype=u8, device=1), xs, w, ws)),
        (TypeError, "codes", lambda: B.fp8_matmul(t(4, 256), xs, w, ws)),
        (ValueError, "w_codes has shape", lambda: B.fp8_matmul(x, xs, t(128, 255, dtype=u8), ws)),
        (ValueError, "scales has shape", lambda: B.fp8_matmul(x, t(4, 3), w, ws, out=out)),
        (ValueError, "w_scales has shape", lambda: B.fp8_matmul(x, xs, w, t(2, 2), out=out)),
        (ValueError, "out has shape", lambda: B.fp8_matmul(x, xs, w, ws, out=t(4, 64, dtype=bf))),
        (TypeError, "out must be", lambda: B.fp8_matmul(x, xs, w, ws, out=t(4, 128, dtype=torch.float64))),
        (ValueError, "two halves", lambda: B.fp8_matmul(x, xs, t(129, 256, dtype=u8), t(2, 2), gated=True)),
        (ValueError, "either out or", lambda: B.fp8_matmul(x, xs, w, ws, gated=True, out=out, out_codes=x, out_scales=xs)),
        (ValueError, "given together", lambda: B.fp8_matmul(x, xs, w, ws, gated=True, out_codes=x)),
        (ValueError, "out_scales has shape",
         lambda: B.fp8_matmul(x, xs, w, ws, gated=True, out_codes=t(4, 64, dtype=u8), out_scales=t(4, 2))),
        (ValueError, "need x_scales", lambda: B.grouped_matmul(x, w3, starts)),
        (ValueError, "scales go", lambda: B.grouped_matmul(t(4, 256, dtype=bf), t(3, 128, 256, dtype=bf), starts, xs, ws3)),
        (TypeError, "weight must be", lambda: B.grouped_matmul(t(4, 256, dtype=bf), t(3, 128, 256, dtype=torch.half), starts)),
        (TypeError, "x must be", lambda: B.grouped_matmul(t(4, 256), t(3, 128, 256), starts)),
        (ValueError, "group_starts has shape", lambda: B.grouped_matmul(x, w3, t(3, dtype=i32), xs, ws3, out=out)),
        (TypeError, "rows must be", lambda: B.grouped_matmul(x, w3, starts, xs, ws3, rows=rows.long())),
        (ValueError, "out has shape", lambda: B.grouped_matmul(x, w3, starts, xs, ws3, rows=rows, out=out)),
        (ValueError, "scoring", lambda: B.route_experts(t(4, 8), 2, t(4, 2, dtype=i32), t(4, 2), t(9, dtype=i32),
                                                        t(8, dtype=i32), t(4, 2, dtype=i32), scoring="relu")),
        (ValueError, "rows has shape", lambda: B.route_experts(t(4, 8), 2, t(4, 2, dtype=i32), t(4, 2), t(9, dtype=i32),
                                                               t(7, dtype=i32), t(4, 2, dtype=i32))),
        (TypeError, "bias", lambda: B.route_experts(t(4, 8), 2, t(4, 2, dtype=i32), t(4, 2), t(9, dtype=i32), t(8, dtype=i32),
                                                    t(4, 2, dtype=i32), bias=t(8, dtype=bf))),
        (TypeError, "add must be", lambda: B.combine_experts(t(8, 64, dtype=bf), t(4, 2, dtype=i32), t(4, 2), add=t(4, 64),
                                                             out=t(4, 64, dtype=bf))),
        (ValueError, "weights has shape", lambda: B.combine_experts(t(8, 64, dtype=bf), t(4, 2, dtype=i32), t(4, 3),
                                                                    out=t(4, 64, dtype=bf))),
    ]:
        if match in ("scales has shape", "out has shape", "w_scales has shape"):
            monkeypatch.setattr(B, "load", lambda: type("Lib", (), {"__getattr__": lambda *a: lambda *b: pytest.fail("the call went on")})())
        with pytest.raises(error, match=match):
            call()
