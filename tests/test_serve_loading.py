"""Attention calls do without the serving library, and checks of its arguments (no GPU needed)."""
import pytest

from scaled_dot_product_bwd_b200 import binding, serve
from scaled_dot_product_bwd_b200.build import build


class Function:
    """A library's function, which remembers its last arguments."""
    def __init__(self):
        self.got = None

    def __call__(self, *args):
        self.got = args


class Library:
    """Any name is a function."""
    def __getattr__(self, name):
        self.__dict__[name] = f = Function()
        return f


@pytest.fixture
def unloaded(monkeypatch):
    build()
    for name in ("_lib", "_bind", "_wait_limit_ns"):
        monkeypatch.setattr(serve, name, None, raising=False)
    yield monkeypatch
    binding.load_library().sdpa_set_wait_limit_ns(2000000000)


def test_the_wait_limit_is_set_without_the_serving_library(unloaded, tmp_path):
    unloaded.setattr(serve, "SERVE_LIB_PATH", str(tmp_path / "missing.so"))
    binding.sdpa_set_wait_limit_ns(2000000000)
    assert serve.read_device_status(None) == 0
    with pytest.raises(RuntimeError):
        serve.load_serve_library()


def test_the_wait_limit_reaches_a_library_loaded_later(unloaded):
    binding.sdpa_set_wait_limit_ns(1500000000)
    library = Library()
    unloaded.setattr(serve.ctypes, "CDLL", lambda path: library)
    serve.load_serve_library()
    assert library.sdpa_serve_set_wait_limit_ns.got == (1500000000,)
    binding.sdpa_set_wait_limit_ns(1600000000)
    assert library.sdpa_serve_set_wait_limit_ns.got == (1600000000,)


def test_a_row_stride_of_zero_passes_the_checks_and_one_below_the_width_does_not():
    """Past the stride, what follows in the checks refuses: a missing workspace, a missing output."""
    import ctypes

    from test_serve_abi import FAKE, NULL, _cache, _rope, _tree
    lib = serve.load_serve_library()
    c = _cache()
    for step, code in ((0, 3), (4, 1)):
        t = _tree(table_b=step)
        assert lib.sdpa_tree_fwd(ctypes.byref(t), ctypes.byref(c), FAKE, None, 0.1, FAKE, FAKE, NULL, 0, None) == code
        assert (lib.sdpa_tree_fwd_workspace_size(ctypes.byref(t), ctypes.byref(c)) > 0) == (step == 0)
    r = _rope(pos_b=0)
    assert lib.sdpa_rope(ctypes.byref(r), FAKE, FAKE, FAKE, NULL, None) == 1      # (for k_out)


def test_append_of_keys_alone_passes_the_checks_of_its_pointers():
    import ctypes

    from test_serve_abi import FAKE, NULL, _cache
    lib = serve.load_serve_library()
    c = _cache()
    call = lambda k, v, T: lib.sdpa_cache_append(ctypes.byref(c), k, v, T, 128, 64, FAKE, None)
    assert call(FAKE, NULL, 1 << 31) == 2                    # (refused for T, after them)
    assert call(NULL, FAKE, 4) == call(NULL, NULL, 4) == call(FAKE, ctypes.c_void_p(0x10008), 4) == 1
