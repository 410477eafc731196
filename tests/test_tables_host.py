"""Weight-table operators, checks that need no GPU: the C entry points refuse
bad arguments before any device call, the workspace size, the binding's types."""
import ctypes

import pytest

import spmv_storage_formats_amd as spmv

INVALID, TOO_LARGE = 1, 5
P = ctypes.c_void_p(4096)    # a pointer that no refused call follows
FP32, FP16, BF16, INT32, INT64 = range(5)


@pytest.fixture(scope="module")
def lib():
    return spmv.load_library()


def test_dtype_codes_match_the_header():
    import os
    import re
    hdr = open(os.path.join(os.path.dirname(spmv.__file__), "..", "include", "spmv.h")).read()
    body = re.search(r"typedef enum spmv_dtype \{(.*?)\}", hdr, re.S).group(1)
    found = {m.group(1): int(m.group(2)) for m in re.finditer(r"SPMV_(\w+) = (\d)", body)}
    assert found == {"FP32": 0, "FP16": 1, "BF16": 2, "INT32": 3, "INT64": 4}
    assert list(spmv.DTYPES.values()) == [0, 1, 2, 3, 4]
    assert spmv.STATUS[9] == "SPMV_ERR_BAD_VALUE"
    assert b"finite" in spmv.load_library().spmv_status_string(9)


@pytest.mark.parametrize("change", [
    {"R": -1}, {"C": -1}, {"group": 0}, {"group": 16}, {"group": 96}, {"group": -128},
    {"group": 192}, {"scale": INT32}, {"scale": 7}, {"weight": INT64}, {"weights": None},
    {"ld": 255}])
def test_build_refusals(lib, change):
    a = dict(R=4, C=256, group=128, zeros=0, scale=FP32, weights=P, ld=256, weight=FP32)
    a.update(change)
    out = ctypes.c_void_p(77)
    assert lib.spmv_quant_build(ctypes.byref(out), a["R"], a["C"], a["group"], a["zeros"],
                                a["scale"], a["weights"], a["ld"], a["weight"], None) == INVALID
    assert out.value is None
    assert lib.spmv_quant_build(None, 4, 256, 128, 0, FP32, P, 256, FP32, None) == INVALID


@pytest.mark.parametrize("change", [
    {"R": -1}, {"C": -1}, {"group": 33}, {"scale": INT64}, {"codes": None}, {"scales": None}])
def test_build_packed_refusals(lib, change):
    a = dict(R=4, C=256, group=64, codes=P, scales=P, scale=BF16)
    a.update(change)
    out = ctypes.c_void_p(77)
    assert lib.spmv_quant_build_packed(ctypes.byref(out), a["R"], a["C"], a["group"], a["codes"],
                                       a["scales"], a["scale"], None, 1, None) == INVALID
    assert out.value is None
    assert lib.spmv_quant_build_packed(None, 4, 256, 64, P, P, BF16, None, 1, None) == INVALID


def test_null_quant_handles(lib):
    n = ctypes.c_size_t()
    info = spmv._QuantInfo()
    assert lib.spmv_quant_run(None, 1, P, 4, FP32, P, 4, FP32, 1, None, 0, None) == INVALID
    assert lib.spmv_quant_run_workspace(None, 1, FP32, ctypes.byref(n)) == INVALID
    assert lib.spmv_quant_lookup(None, 1, P, INT32, 1.0, P, 4, FP32, None) == INVALID
    assert lib.spmv_quant_get_info(None, ctypes.byref(info)) == INVALID
    assert lib.spmv_quant_array_bytes(None, 0, ctypes.byref(n)) == INVALID
    assert lib.spmv_quant_export(None, 0, P, 4) == INVALID
    assert lib.spmv_quant_destroy(None) == 0


@pytest.mark.parametrize("n,status", [
    (2**31 - 50, 0), (2**31 - 49, 0), (2**31 - 48, TOO_LARGE), (2**31 - 1, TOO_LARGE)])
def test_products_refuse_vectors_that_a_pass_would_wrap(lib, n, status):
    """The last pass of up to 48 vectors begins at most at n - 1, and the kernels form the
    index of its last vector, there or not, in 32 bits.  The handle is a zeroed one: an empty
    matrix, for which an accepted call does nothing."""
    empty = ctypes.create_string_buffer(512)
    size = ctypes.c_size_t(7)
    assert lib.spmv_quant_run_workspace(empty, n, BF16, ctypes.byref(size)) == status
    assert size.value == (7 if status else 0)
    assert lib.spmv_quant_run(empty, n, P, 1, BF16, P, 1, BF16, 1, None, 0, None) == status
    if status == 0:
        assert n - 1 + 48 <= 2**31 - 1


@pytest.mark.parametrize("change", [
    {"V": -1}, {"D": -1}, {"n": -1}, {"table_dtype": INT32}, {"id": FP32}, {"out_dtype": INT64},
    {"table": None}, {"ids": None}, {"out": None}, {"table_ld": 7}, {"out_ld": 7}])
def test_lookup_refusals(lib, change):
    a = dict(V=10, D=8, table=P, table_ld=8, table_dtype=BF16, n=3, ids=P, id=INT32, out=P,
             out_ld=8, out_dtype=FP32)
    a.update(change)
    assert lib.spmv_lookup(a["V"], a["D"], a["table"], a["table_ld"], a["table_dtype"], a["n"],
                           a["ids"], a["id"], 1.0, a["out"], a["out_ld"], a["out_dtype"],
                           None) == INVALID


def test_nothing_to_look_up_is_no_error(lib):
    assert lib.spmv_lookup(10, 8, P, 8, FP32, 0, None, INT32, 1.0, None, 8, FP32, None) == 0
    assert lib.spmv_lookup(10, 0, P, 0, FP32, 5, P, INT32, 1.0, None, 0, FP32, None) == 0
    assert lib.spmv_lookup_grad(0, 8, 5, P, INT32, P, 8, FP32, 1.0, 0, None, 8, FP32, None, 0,
                                None) == 0
    assert lib.spmv_lookup_grad(8, 0, 5, P, INT32, P, 0, FP32, 1.0, 0, None, 0, FP32, None, 0,
                                None) == 0


@pytest.mark.parametrize("change,status", [
    ({"V": -1}, INVALID), ({"D": -1}, INVALID), ({"n": -1}, INVALID), ({"n": 2**31}, TOO_LARGE),
    ({"id": BF16}, INVALID), ({"grad_dtype": INT32}, INVALID), ({"dtype": INT64}, INVALID),
    ({"ids": None}, INVALID), ({"grad": None}, INVALID), ({"out": None}, INVALID),
    ({"grad_ld": 7}, INVALID), ({"ld": 7}, INVALID), ({"ws": None}, INVALID),
    ({"ws": ctypes.c_void_p(4100)}, INVALID), ({"short": 1}, INVALID)])
def test_lookup_grad_refusals(lib, change, status):
    a = dict(V=10, D=8, n=300, ids=P, id=INT64, grad=P, grad_ld=8, grad_dtype=FP16, out=P, ld=8,
             dtype=FP32, ws=P, short=0)
    a.update(change)
    n = spmv.lookup_grad_workspace(300, 10, 8)
    assert lib.spmv_lookup_grad(a["V"], a["D"], a["n"], a["ids"], a["id"], a["grad"],
                                a["grad_ld"], a["grad_dtype"], 1.0, 0, a["out"], a["ld"],
                                a["dtype"], a["ws"], n - a["short"], None) == status


def test_workspace_size(lib):
    n = ctypes.c_size_t()
    assert lib.spmv_lookup_grad_workspace(10, 8, 2**31, ctypes.byref(n)) == TOO_LARGE
    assert lib.spmv_lookup_grad_workspace(10, 8, -1, ctypes.byref(n)) == INVALID
    assert lib.spmv_lookup_grad_workspace(10, 8, 5, None) == INVALID
    assert spmv.lookup_grad_workspace(0, 10, 8) == 0
    assert spmv.lookup_grad_workspace(5, 0, 8) == 0
    sizes = [spmv.lookup_grad_workspace(k, 1000, 64) for k in (1, 100, 10_000, 1_000_000)]
    assert sizes == sorted(sizes) and sizes[0] > 0
    # two copies of (key, position) are the least a sort that ping-pongs keeps
    assert sizes[-1] >= 16 * 1_000_000
    with pytest.raises(spmv.SpmvError):
        spmv.lookup_grad_workspace(-1, 10, 8)


def test_committed_profile_matches_the_kernel_sources():
    """The kernel times and counters of profiles/weight_tables_kernel_trace.md were taken on
    the committed code: the hash that it carries is that of the sources that the weight
    tables' kernels are compiled from, comments and whitespace removed."""
    import hashlib
    import os
    import re
    package = os.path.dirname(spmv.__file__)
    h = hashlib.sha256()
    for f in ("internal.h", "tables.h", "quant.hip", "quant_product.h", "quant_run_bf16.hip",
              "quant_run_fp16.hip", "quant_run_fp32.hip", "lookup.hip"):
        text = open(os.path.join(package, "csrc", f), encoding="utf-8").read()
        text = re.sub(r"//[^\n]*", " ", re.sub(r"/\*.*?\*/", " ", text, flags=re.S))
        h.update(" ".join(text.split()).encode())
    profile = open(os.path.join(package, "..", "profiles", "weight_tables_kernel_trace.md"),
                   encoding="utf-8").read()
    assert f"kernel_source_sha: {h.hexdigest()[:16]}" in profile


def test_binding_rejects_host_tensors():
    torch = pytest.importorskip("torch")
    w = torch.zeros(4, 64)
    ids = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(TypeError):
        spmv.build_quant(w)
    with pytest.raises(TypeError):
        spmv.build_quant_packed(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 1), 64)
    with pytest.raises(TypeError):
        spmv.lookup(w, ids)
    with pytest.raises(TypeError):
        spmv.lookup_grad(torch.zeros(3, 64), ids, 10)


def test_product_refuses_what_is_no_tensor():
    torch = pytest.importorskip("torch")
    q = spmv.QuantHandle.__new__(spmv.QuantHandle)     # refused before the handle is used
    q._ptr, q.device = P, torch.device("cuda:0")
    try:
        for x, y in ((None, None), ([1.0], torch.zeros(1)), (torch.zeros(1), 3)):
            with pytest.raises(TypeError):
                q.run(x, y)
    finally:
        q._ptr = None


def test_binding_refuses_sizes_beyond_int32():
    """Sizes that an int32 argument would wrap (to 5 rows, a group of 32) are refused."""
    torch = pytest.importorskip("torch")
    wrap = 2**32 + 5
    many = torch.zeros(1, 1).expand(wrap, 1)
    ids = torch.zeros(3, dtype=torch.int64)
    for call in (lambda: spmv.lookup_grad_workspace(5, wrap, 8),
                 lambda: spmv.lookup_grad_workspace(5, 8, wrap),
                 lambda: spmv.lookup_grad_workspace(wrap, 8, 8),
                 lambda: spmv.lookup(many, ids),
                 lambda: spmv.build_quant(many),
                 lambda: spmv.build_quant(torch.zeros(4, 64), group_size=2**32 + 32),
                 lambda: spmv.build_quant_packed(None, None, wrap),
                 lambda: spmv.build_quant_packed(None, None, 64, group_size=2**32 + 32)):
        with pytest.raises(spmv.SpmvError) as e:
            call()
        assert e.value.status == TOO_LARGE


def test_binding_refuses_sizes_below_int32():
    """Sizes that an int32 argument would wrap from below (to 5 tokens, 8 rows, a group of 32)
    are refused as negative ones are; so is a count of tokens that 64 bits would wrap."""
    torch = pytest.importorskip("torch")
    wrap = -2**32 + 8
    for call in (lambda: spmv.lookup_grad_workspace(5, wrap, 8),
                 lambda: spmv.lookup_grad_workspace(5, 8, wrap),
                 lambda: spmv.lookup_grad_workspace(-2**64 + 5, 8, 8),
                 lambda: spmv.build_quant(torch.zeros(4, 64), group_size=-2**32 + 32)):
        with pytest.raises(spmv.SpmvError) as e:
            call()
        assert e.value.status == INVALID
    with pytest.raises(spmv.SpmvError) as e:
        spmv.lookup_grad_workspace(2**64 + 5, 8, 8)
    assert e.value.status == TOO_LARGE


def test_binding_overlap_rule():
    """Spans that meet are refused; column ranges of one buffer side by side are not."""
    torch = pytest.importorskip("torch")
    buf = torch.zeros(6, 32)
    spmv._apart(buf[:, :16], buf[:, 16:], "halves")
    spmv._apart(buf[:3], buf[3:], "rows")
    spmv._apart(buf[:0], buf, "nothing")
    for a, b in ((buf, buf), (buf[:, :17], buf[:, 16:]), (buf[:4], buf[3:]),
                 (buf[:, 16:], buf[:, 8:20]), (buf.view(-1), buf[2])):
        with pytest.raises(ValueError):
            spmv._apart(a, b, "these")
