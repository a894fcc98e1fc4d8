"""CPU-side checks of the paged cache of 8-bit codes: metadata errors come before any GPU work, and the binding refuses
scales that do not belong to their cache."""
import pytest

torch = pytest.importorskip("torch")

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from tests.test_kv_abi_cpu import FAKE, INVALID, OVERFLOW, UNSUPPORTED, append, attention, cache, lib, step  # noqa: E402,F401
from tests.test_kv_binding_cpu import Tensor, f32, i32, rows  # noqa: E402
from tests.test_kv_binding_cpu import lib as fake  # noqa: E402,F401

E4M3 = torch.float8_e4m3fn


def codes(**kw):
    d = dict(dtype=mnb.E4M3, k_scale=FAKE, v_scale=FAKE, scale_page_stride=8, scale_head_stride=1, scale_block=16)
    d.update(kw)
    return cache(**d)


BAD = [(dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(scale_block=0), INVALID),
       (dict(scale_block=8, scale_head_stride=1), INVALID), (dict(scale_page_stride=0), INVALID),
       (dict(scale_block=4), UNSUPPORTED), (dict(scale_block=12), UNSUPPORTED), (dict(scale_block=32), UNSUPPORTED),
       (dict(page_size=256, scale_block=256), UNSUPPORTED), (dict(head_dim=104, token_stride=112), UNSUPPORTED),
       (dict(token_stride=136), UNSUPPORTED), (dict(k_scale=FAKE + 2), UNSUPPORTED), (dict(v_scale=FAKE + 1), UNSUPPORTED),
       (dict(k=FAKE + 8), UNSUPPORTED), (dict(scale_page_stride=1 << 61), OVERFLOW)]


@pytest.mark.parametrize("bad,code", BAD)
def test_cache_errors(lib, bad, code):  # noqa: F811
    assert append(lib, c=codes(**bad)) == code
    assert attention(lib, c=codes(**bad)) == code


def test_any_float_rows_go_over_codes(lib):  # noqa: F811
    for dt in (0, 1, 2):
        assert append(lib, c=codes(), s=step(tokens=0), dt=dt) == 0
        assert attention(lib, c=codes(), s=step(tokens=0), dt=dt) == 0
    assert append(lib, c=codes(), dt=mnb.E4M3) == INVALID
    assert attention(lib, c=codes(), dt=mnb.E4M3) == INVALID
    assert append(lib, c=cache(), dt=1) == UNSUPPORTED  # a 16-bit cache takes its own type or fp32


def test_scales_of_one_page_or_head_need_no_stride(lib):  # noqa: F811
    assert append(lib, c=codes(num_pages=1, scale_page_stride=0), s=step(tokens=0)) == 0
    assert append(lib, c=codes(kv_heads=1, scale_head_stride=0), s=step(tokens=0)) == 0


def pages(dtype=E4M3, device=0, dim=64):
    return Tensor((9, 2, 16, dim), dtype, device)


def test_binding_of_scales(fake):  # noqa: F811
    d = mnb.kv_cache(pages(), pages(), f32(9, 2, 2), f32(9, 2, 2))
    assert (d.dtype, d.scale_block, d.scale_page_stride, d.scale_head_stride) == (mnb.E4M3, 8, 4, 2)
    assert mnb.kv_cache(pages(torch.float16), pages(torch.float16)).k_scale is None
    for bad in ((None, None), (f32(9, 2, 2), None), (None, f32(9, 2, 2)), (f32(9, 2, 3), f32(9, 2, 3)), (f32(9, 2), f32(9, 2)),
                (f32(8, 2, 2), f32(8, 2, 2)), (f32(9, 2, 2), f32(9, 2, 1)), (f32(9, 2, 2), f32(9, 2, 2, device=1)),
                (f32(9, 2, 0), f32(9, 2, 0))):
        with pytest.raises(ValueError):
            mnb.kv_cache(pages(), pages(), *bad)
    with pytest.raises(ValueError):
        mnb.kv_cache(pages(torch.float16), pages(torch.float16), f32(9, 2, 2), f32(9, 2, 2))
    with pytest.raises(TypeError):
        mnb.kv_cache(pages(), pages(), i32(9, 2, 2), i32(9, 2, 2))
    with pytest.raises(TypeError):
        mnb.kv_cache(pages(torch.uint8), pages(torch.uint8))
    s = mnb.kv_step(i32(3), i32(3, 4))
    mnb.kv_append(d, s, rows(4), rows(2), rows(2), rows(4))
    assert fake.calls.pop()[0] == "kv_append"
    with pytest.raises(TypeError):  # codes are not rows
        mnb.kv_append(d, s, Tensor((3, 4, 64), E4M3), Tensor((3, 2, 64), E4M3), Tensor((3, 2, 64), E4M3), Tensor((3, 4, 64), E4M3))
    with pytest.raises(ValueError):
        mnb.kv_append(mnb.kv_cache(pages(device=1), pages(device=1), f32(9, 2, 2, device=1), f32(9, 2, 2, device=1)), s, rows(4),
                      rows(2), rows(2), rows(4))
    assert fake.calls == []
