"""Work handles and the training operators without a device: refusals that come before any
CUDA call, and the binding's structs against the header's (CPU)."""
import ctypes
import os
import re

import pytest

import server_side_fedavg_gb300 as fa

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fedavg.h")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fa.lib()


def test_null_handles_are_refused(lib):
    assert lib.fa_work_open(None, None) == fa.FA_ERR_ARG
    assert lib.fa_work_close(None) == fa.FA_OK
    assert lib.fa_work_sync(None) == fa.FA_ERR_ARG
    assert lib.fa_work_get_stats(None, None) == fa.FA_ERR_ARG
    assert lib.fa_product(None, None, None) == fa.FA_ERR_ARG
    assert lib.fa_product_backward(None, None, None) == fa.FA_ERR_ARG
    assert lib.fa_distill_loss(None, None, None) == fa.FA_ERR_ARG
    assert lib.fa_distill_grad(None, None, None) == fa.FA_ERR_ARG
    assert fa.fa_work_last_error(None) == ""


def test_bad_options_are_refused(lib):
    w = ctypes.c_void_p()
    for opts in (fa.fa_work_opts(4, 0, 0, 0, 0), fa.fa_work_opts(ctypes.sizeof(fa.fa_work_opts), 0, 0, 1, 0),
                 fa.fa_work_opts(ctypes.sizeof(fa.fa_work_opts), 0, 1 << 41, 0, 0)):
        assert lib.fa_work_open(ctypes.byref(opts), ctypes.byref(w)) == fa.FA_ERR_ARG and w.value is None


def test_lists_of_different_lengths_are_refused():
    with pytest.raises(ValueError, match="lengths differ"):
        fa.distill_lists([0, 0], [0, 0], [4], [1.0, 1.0])


def test_structs_have_the_headers_fields():
    """Each struct's field names and types in order, from the header's text."""
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    ctype = {"uint32_t": ctypes.c_uint32, "int32_t": ctypes.c_int32, "uint64_t": ctypes.c_uint64,
             "double": ctypes.c_double}
    for name in ("fa_work_opts", "fa_work_stats", "fa_product_args", "fa_product_backward_args", "fa_distill_client",
                 "fa_distill_args"):
        body = re.search(r"typedef struct \{([^{}]*)\} " + name + r";", text).group(1)
        want = []
        for decl in filter(None, (d.strip() for d in body.split(";"))):
            pointer = "*" in decl
            words = decl.replace("const ", "").replace("*", " ")
            kind, names = words.split(None, 1)
            want += [(n.strip(), ctypes.c_void_p if pointer else ctype[kind]) for n in names.split(",")]
        assert list(getattr(fa, name)._fields_) == want, name
