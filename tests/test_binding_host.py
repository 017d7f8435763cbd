"""What the Python binding hands to the library, seen through stand-ins for
torch's CUDA part and for the library (no GPU needed)."""
import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_pa_gb300 as pa


class Tensor:
    """A CUDA tensor as far as the binding looks; `home`: the stream whose memory it is."""

    def __init__(self, shape, dtype, home="caller", device=0):
        self.shape = torch.Size((shape,) if isinstance(shape, int) else shape)
        self.dtype, self.home = dtype, home
        self.device = types.SimpleNamespace(type="cuda", index=device)
        self.is_cuda, self.used_by = True, []

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def get_device(self):
        return self.device.index

    def data_ptr(self):
        return id(self)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    def record_stream(self, stream):
        self.used_by.append(stream)


class Torch:
    """torch, its tensors and streams stood in for."""

    def __init__(self, device=0):
        self.stream, self.made, self.device = "current", [], device
        outer = self

        class Cuda:
            @staticmethod
            @contextlib.contextmanager
            def stream(s):
                before, outer.stream = outer.stream, s
                yield
                outer.stream = before

            @staticmethod
            def device_count():
                return 2

            @staticmethod
            def current_stream(device=None):
                return outer.stream

        self.cuda = Cuda
        self._C = types.SimpleNamespace(_cuda_getCurrentRawStream=lambda i: 1000 + i,
                                        _cuda_getDevice=lambda: outer.device)

    def __getattr__(self, name):
        return getattr(torch, name)

    def empty(self, *shape, dtype=None, device=None):
        shape = shape[0] if len(shape) == 1 else shape
        self.made.append(Tensor(shape, dtype, self.stream))
        return self.made[-1]


class Library:
    """Accepts every call."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def call(*args):
            self.calls.append((name, args))
            return 4096 if name.endswith("_size") else 0
        return call


@pytest.fixture
def fake(monkeypatch):
    t, lib = Torch(), Library()
    monkeypatch.setattr(pa, "_torch_module", t)
    monkeypatch.setattr(pa, "_lib", lib)
    monkeypatch.setattr(pa, "_DTYPE_CODES", {})
    monkeypatch.setattr(pa, "_several_devices", None)
    return types.SimpleNamespace(torch=t, lib=lib)


def _calls():
    h, i32, i64, f32 = torch.float16, torch.int32, torch.int64, torch.float32
    q, new = Tensor((2, 8, 64), h), Tensor((2, 4, 64), h)
    pool = Tensor((9, 4, 16, 64), h)
    tab, lens, qsl = Tensor((2, 4), i32), Tensor(2, i32), Tensor(3, i32)
    sc, lse = Tensor((2, 4, 64), f32), Tensor((2, 8), f32)
    rot = types.SimpleNamespace(num_axes=1, _ptr=1)
    return {
        "rotary": lambda **kw: pa.rotary_cache_write(q, new, new, Tensor(2, i64), rot, pool, pool, Tensor(2, i64), **kw),
        "decode": lambda **kw: pa.decode_attention(q, pool, pool, tab, lens, 64, 0.1, **kw),
        "contiguous": lambda **kw: pa.decode_attention_contiguous(q, Tensor((2, 4, 64, 64), h), Tensor((2, 4, 64, 64), h),
                                                                  lens, 64, 0.1, **kw),
        "scored": lambda **kw: pa.decode_attention_scored(q, pool, pool, tab, lens, 64, 0.1, sc, **kw),
        "prefill": lambda **kw: pa.prefill_attention(q, pool, pool, tab, qsl, lens, 2, 64, 0.1, **kw),
        "prompt scores": lambda **kw: pa.prefill_scores(q, lse, pool, tab, qsl, lens, 2, 64, 0.1, sc, **kw),
        "evict": lambda **kw: pa.evict_tokens([pool], [pool], [sc], tab, lens, lens, 64, 32, **kw),
    }


@pytest.mark.parametrize("name", list(_calls()))
def test_what_a_call_allocates_belongs_to_its_stream(fake, name):
    """Memory of the current stream may still be in use there, and goes back to it when the
    call returns: the call's kernels, on another stream, must not get it."""
    side = types.SimpleNamespace(cuda_stream=7)
    got = _calls()[name](stream=side)
    assert all(t.home is side for t in fake.torch.made)
    assert fake.lib.calls[-1][1][-1] == 7
    if got in fake.torch.made:  # the current stream will use it
        assert got.used_by == ["current"]
    del fake.torch.made[:]
    _calls()[name]()
    assert all(t.home == "current" for t in fake.torch.made)
    assert fake.lib.calls[-1][1][-1] == 1000


@pytest.mark.parametrize("how", ["copy", "deepcopy", "pickle"])
def test_a_copied_rotary_has_frequencies_of_its_own(fake, how):
    """A module that holds one may be copied, and outlive the original."""
    import copy
    import ctypes
    import pickle
    rot = pa.Rotary([0.5] * 8)
    rot._struct.turns[3] = 77
    again = {"copy": copy.copy, "deepcopy": copy.deepcopy,
             "pickle": lambda r: pickle.loads(pickle.dumps(r))}[how](rot)
    h, i64 = torch.float16, torch.int64
    q, new, pool = Tensor((2, 8, 64), h), Tensor((2, 4, 64), h), Tensor((9, 4, 16, 64), h)
    pa.rotary_cache_write(q, new, new, Tensor(2, i64), again, pool, pool, Tensor(2, i64))
    name, args = fake.lib.calls[-1]
    assert name == "pa_rotary_cache_write" and args[9] == ctypes.addressof(again._struct)
    assert again._struct.turns[3] == 77 and again.rotary_dim == rot.rotary_dim


@pytest.mark.parametrize("name", list(_calls()))
def test_tensors_on_another_device_than_the_current_one_are_refused(fake, name):
    """The library launches on the current device; the default stream has the same handle on all."""
    fake.torch.device = 1
    for kw in ({}, {"stream": types.SimpleNamespace(cuda_stream=7)}):
        with pytest.raises(ValueError, match="current device"):
            _calls()[name](**kw)
    assert all(n.endswith("_size") for n, _ in fake.lib.calls)


def test_prompt_scores_take_no_memory(fake):
    _calls()["prompt scores"]()
    assert not fake.torch.made
    assert fake.lib.calls[-1][1][-4:-2] == (None, 0)
    ws = Tensor(256, torch.uint8)
    _calls()["prompt scores"](workspace=ws)
    assert fake.lib.calls[-1][1][-4:-2] == (ws.data_ptr(), 256)


def test_the_current_stream_given_by_name_is_the_current_stream(fake):
    side = types.SimpleNamespace(cuda_stream=1000)  # the current stream's handle
    for call in _calls().values():
        call(stream=side)
        assert fake.lib.calls[-1][1][-1] == 1000
    assert all(t.home == "current" and not t.used_by for t in fake.torch.made)


def test_a_swap_between_pinned_pools_needs_no_device(fake):
    """Nothing to move, and no tensor of the call on a GPU."""
    def host(shape, dtype):
        t = Tensor(shape, dtype)
        t.is_cuda, t.is_pinned = False, lambda: True
        return t
    pool = host((9, 4, 16, 64), torch.float16)
    pa.swap_blocks([pool], [pool], [pool], [pool], host((0, 2), torch.int64), stream=types.SimpleNamespace(cuda_stream=7))
    assert fake.lib.calls[-1][0] == "pa_swap_blocks" and fake.lib.calls[-1][1][-1] == 7
