"""The binding of the paged-cache and draft-verification calls without a GPU: stand-ins
for CUDA tensors, and a stand-in for the library that notes its calls."""
import ctypes
import gc
import weakref

import pytest

torch = pytest.importorskip("torch")

import qmoe_mnb_matmul_gb300 as mnb  # noqa: E402
from qmoe_mnb_matmul_gb300 import _binding  # noqa: E402


class Tensor:
    """What the binding asks of a CUDA tensor."""

    def __init__(self, shape, dtype=torch.bfloat16, device=0):
        self.shape, self.dtype, self.index = torch.Size(shape), dtype, device
        self.is_cuda = device >= 0
        self._stride = torch.empty(shape, device="meta").stride()

    def stride(self, i=None):
        return self._stride if i is None else self._stride[i]

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    def data_ptr(self):
        return 0x10000

    def element_size(self):
        return self.dtype.itemsize

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize


class Library:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    library = Library()
    monkeypatch.setattr(_binding, "load_library", lambda path=None: library)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 1000 + device, raising=False)
    return library


def i32(*shape, device=0):
    return Tensor(shape, torch.int32, device)


def f32(*shape, device=0):
    return Tensor(shape, torch.float32, device)


def cache(device=0):
    return mnb.kv_cache(Tensor((9, 2, 16, 64), device=device), Tensor((9, 2, 16, 64), device=device))


def step(device=0):
    return mnb.kv_step(i32(3, device=device), i32(3, 4, device=device))


def rows(heads, device=0):
    return Tensor((3, heads, 64), device=device)


def append(c=None, s=None, rope=None, q=None, k=None, v=None, out=None, **kw):
    return mnb.kv_append(c or cache(), s or step(), q or rows(4), k or rows(2), v or rows(2), out or rows(4), rope, **kw)


def attend(c=None, s=None, q=None, out=None, ws=None, **kw):
    return mnb.kv_attention(c or cache(), s or step(), q or rows(4), out or rows(4), ws or Tensor((1 << 20,), torch.uint8), **kw)


@pytest.mark.parametrize("kind", ["cache", "step", "rope"])
def test_a_dropped_descriptor_frees_its_tensors_at_once(lib, kind):
    gc.collect()
    gc.disable()
    try:
        t = {"cache": Tensor((9, 2, 16, 64)), "step": i32(3), "rope": f32(64)}[kind]
        held = weakref.ref(t)
        d = {"cache": lambda: mnb.kv_cache(t, t), "step": lambda: mnb.kv_step(t, i32(3, 4)),
             "rope": lambda: mnb.kv_rope(q_norm=t)}[kind]()
        t = None
        assert held() is not None  # the descriptor keeps what it points to
        d = None  # noqa: F841
        assert held() is None
    finally:
        gc.enable()


def test_a_descriptor_that_the_caller_builds(lib):
    c = mnb.KvCacheDesc(k=0x10000, v=0x20000, num_pages=9, page_stride=2048, head_stride=1024, token_stride=64, page_size=16,
                        kv_heads=2, head_dim=64, dtype=mnb.BF16)
    s = mnb.KvStepDesc(seq_lens=0x10000, new_start=None, page_table=0x20000, table_stride=4, batch=3, tokens=3, max_new=1,
                       max_pages=4)
    r = mnb.KvRopeDesc(cos_sin=0x10000, max_pos=64, rot_dim=64, eps=1e-6)
    append(c, s, r)
    attend(c, s)
    assert [name for name, _ in lib.calls] == ["kv_append", "kv_attention"]
    at = lambda x: x if isinstance(x, int) else ctypes.cast(x, ctypes.c_void_p).value  # noqa: E731
    assert [at(x) for x in lib.calls[0][1][:3]] == [ctypes.addressof(d) for d in (c, s, r)]
    assert [at(x) for x in lib.calls[1][1][:2]] == [ctypes.addressof(d) for d in (c, s)]


def test_norms_have_one_weight_per_element_of_a_head(lib):
    """The kernel reads head_dim (64) weights of each norm that is given."""
    append(rope=mnb.kv_rope(q_norm=f32(64), k_norm=f32(64)))
    append(rope=mnb.kv_rope(k_norm=f32(64)))
    append(rope=mnb.kv_rope(f32(100, 32)))
    assert len(lib.calls) == 3
    for bad in (dict(q_norm=f32(32)), dict(k_norm=f32(128)), dict(q_norm=f32(32), k_norm=f32(32)), dict(k_norm=f32(0))):
        with pytest.raises(ValueError):
            append(rope=mnb.kv_rope(**bad))
    for bad in (dict(q_norm=f32(64), k_norm=f32(32)), dict(q_norm=f32(32), k_norm=f32(64))):
        with pytest.raises(ValueError):
            append(rope=mnb.kv_rope(**bad))
    assert len(lib.calls) == 3


def verify(device=0, **kw):
    t = dict(target=f32(2, 4, 50, device=device), draft=f32(2, 3, 50, device=device), draft_tokens=i32(2, 3, device=device),
             uniforms=f32(2, 4, device=device), tokens=i32(2, 4, device=device), accepted=i32(2, device=device),
             n_drafts=i32(2, device=device))
    t.update(kw)
    return mnb.draft_verify(t["target"], t["draft"], t["draft_tokens"], t["uniforms"], t["tokens"], t["accepted"],
                            n_drafts=t["n_drafts"])


@pytest.mark.parametrize("where", [1, -1])  # another GPU, the host
def test_every_tensor_is_on_the_current_device(lib, monkeypatch, where):
    """The library launches on the current device, whatever device the tensors are on."""
    far = rows(2, device=where)
    for bad in (dict(q=rows(4, device=where)), dict(k=far), dict(v=far), dict(out=rows(4, device=where))):
        with pytest.raises(ValueError):
            append(**bad)
    for bad in (dict(q=rows(4, device=where)), dict(out=rows(4, device=where)), dict(ws=Tensor((1 << 20,), torch.uint8, where)),
                dict(lse=f32(3, 4, device=where))):
        with pytest.raises(ValueError):
            attend(**bad)
    for name in ("draft_tokens", "tokens"):
        with pytest.raises(ValueError):
            verify(**{name: i32(2, 3 if name == "draft_tokens" else 4, device=where)})
    for bad in (dict(target=f32(2, 4, 50, device=where)), dict(draft=f32(2, 3, 50, device=where)),
                dict(uniforms=f32(2, 4, device=where)), dict(accepted=i32(2, device=where)), dict(n_drafts=i32(2, device=where))):
        with pytest.raises(ValueError):
            verify(**bad)
    # descriptors: tensors of one device, which is the current one at the call
    for make in (lambda: mnb.kv_cache(Tensor((9, 2, 16, 64)), Tensor((9, 2, 16, 64), device=where)),
                 lambda: mnb.kv_step(i32(3), i32(3, 4, device=where)), lambda: mnb.kv_step(i32(3, device=where), i32(3, 4)),
                 lambda: mnb.kv_step(i32(3), i32(3, 4), new_start=i32(4, device=where), tokens=3),
                 lambda: mnb.kv_rope(f32(100, 64), q_norm=f32(64, device=where)),
                 lambda: mnb.kv_rope(f32(100, 64, device=where), k_norm=f32(64))):
        with pytest.raises(ValueError):
            make()
    if where > 0:
        for bad in (dict(c=cache(where)), dict(s=step(where)), dict(rope=mnb.kv_rope(q_norm=f32(64, device=where)))):
            with pytest.raises(ValueError):
                append(**bad)
        for bad in (dict(c=cache(where)), dict(s=step(where))):
            with pytest.raises(ValueError):
                attend(**bad)
    assert lib.calls == []
    if where > 0:  # and with that device current, all of them run, on its stream
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: where, raising=False)
        append(cache(where), step(where), mnb.kv_rope(q_norm=f32(64, device=where)), rows(4, where), rows(2, where),
               rows(2, where), rows(4, where))
        attend(cache(where), step(where), rows(4, where), rows(4, where), Tensor((1 << 20,), torch.uint8, where))
        verify(where)
        assert [args[-1] for _, args in lib.calls] == [1000 + where] * 3


def products(where):
    """Every other call of the binding that launches, with its first tensor on device `where`."""
    u8 = lambda *shape: Tensor(shape, torch.uint8)  # noqa: E731
    A, W, s, Y = f32(1, 64, device=where), u8(32, 2, 16), f32(32, 2), f32(1, 32)
    qm = (f32(1, 8), 2, True, u8(8, 64, 32), f32(8, 64, 2), None, 4, u8(8, 64, 16), f32(8, 64, 1), None, 4, 32, 32, f32(1, 64))
    Wd = Tensor((32, 2, 16), torch.uint8, where)
    yield lambda: mnb.mnb_matmul(A, W, s, None, 32, 4, 32, Y, workspace=u8(64))
    yield lambda: mnb.mnb_matmul_int8a(A, W, s, None, 32, 4, 32, Y)
    yield lambda: mnb.mnb_gate_up_swiglu(A, W, s, None, 16, 4, 32, Y)
    yield lambda: mnb.mnb_prepack(Wd, s, None, 32, 64, 4, 32, u8(4096))
    yield lambda: mnb.mnb_matmul_prepacked(A, mnb.PrepackedDesc(), u8(4096), Y)
    yield lambda: mnb.qmoe_forward(A, *qm, u8(1 << 20))
    yield lambda: mnb.qmoe_forward_ex(A, *qm, u8(1 << 20))
    yield lambda: mnb.qmoe_forward_static(A, *qm)
    yield lambda: mnb.qmoe_route(f32(1, 8, device=where), 2, True, i32(1, 2), f32(1, 2))
    yield lambda: mnb.qmoe_permute(i32(1, 2, device=where), 8, i32(8), i32(9), i32(2))
    yield lambda: mnb.mnb_unpack_codes(Wd, 32, 64, 4, 32, u8(32, 64))
    yield lambda: mnb.mnb_pack_codes(Tensor((32, 64), torch.uint8, where), 32, 64, 4, 32, u8(32, 2, 16))
    yield lambda: mnb.mnb_quantize_int3(A, 32, mnb.F32, u8(1, 2, 12), f32(1, 2))


def test_the_other_calls_do_not_launch_for_tensors_of_another_device(lib, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    calls = list(products(1))
    for call in calls:
        with pytest.raises(ValueError):
            call()
    assert lib.calls == []
    for call in products(0):
        call()
    assert len(lib.calls) == len(calls)
    mnb.qmoe_route(0x10000, 2, True, 0x20000, 0x30000, T=1, E=8)  # raw pointers are the caller's
    assert len(lib.calls) == len(calls) + 1
