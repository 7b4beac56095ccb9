"""Rotary positions, group norm and orthogonalised weight steps without a device (CPU, fakes of the
runtime and of the launches): what is refused, which overlaps are taken, what follows a failure; and
the binding's structs against the header's."""
import ctypes
import math
import os
import re

import pytest

import server_side_fedavg_gb300 as fa
from tests.step_shim import FAR, Step, norm, norm_backward, ortho, rotary

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "fedavg.h")
ARG, RANGE, DTYPE = fa.FA_ERR_ARG, fa.FA_ERR_RANGE, fa.FA_ERR_DTYPE
INF, NAN, HUGE = math.inf, math.nan, 1 << 41


@pytest.fixture(scope="module")
def step():
    s = Step()
    yield s
    s.close()


def check(step, name, make, cases):
    assert step.call(name, make()) == fa.FA_OK, step.error()
    for kw, status in cases:
        step.L.ss_reset(0)
        assert step.call(name, make(**kw)) == status, (kw, step.error())
        assert status == fa.FA_OK or step.L.ss_launches() == 0, kw


def test_rotary(step):
    check(step, "fa_rotary", rotary, [
        ({"size": 8}, ARG), ({"flags": 4}, ARG), ({"dtype": 7}, DTYPE), ({"scale": NAN}, ARG), ({"scale": -INF}, ARG),
        ({"r": 0}, RANGE), ({"r": 7}, RANGE), ({"r": 66}, RANGE), ({"dim": 1024, "r": 514}, RANGE), ({"dim": 70000}, RANGE),
        ({"qh": 70000}, RANGE), ({"seq": 1 << 31}, RANGE), ({"batch": 1 << 16, "seq": 1 << 15}, RANGE), ({"turns": False}, ARG),
        ({"position": None, "first": -1}, RANGE), ({"position": None, "first": 1 << 62}, RANGE), ({"position": FAR[4] + 2}, ARG),
        ({"q": None}, ARG), ({"qo": None}, ARG), ({"ko": None}, ARG), ({"q": FAR[0] + 1}, ARG),
        ({"kh": 0, "k": None, "ko": None}, fa.FA_OK), ({"batch": 0}, fa.FA_OK), ({"seq": 0, "q": None}, fa.FA_OK),
        ({"qh": 0, "kh": 0, "q": None, "qo": None, "k": None, "ko": None}, fa.FA_OK),
        ({"qs": (HUGE, 256, 64)}, RANGE), ({"qos": (0, 256, 64)}, RANGE), ({"qos": (8 * 256, 255, 64)}, RANGE),
        ({"qs": (0, 64, 0)}, fa.FA_OK), ({"qs": (8 * 64, 64, 0)}, fa.FA_OK), ({"batch": 1, "qos": (0, 256, 64)}, fa.FA_OK),
        ({"seq": (1 << 31) - 1, "batch": 1, "qs": ((1 << 40) - 1, (1 << 40) - 1, 64)}, RANGE),      # beyond any address
        # overlaps: an output may be its input, with the same strides, and nothing else
        ({"qo": FAR[0]}, fa.FA_OK), ({"qo": FAR[0], "qos": (8 * 512, 512, 64)}, ARG), ({"qo": FAR[0] + 128}, ARG), ({"qo": FAR[2]}, ARG),
        ({"ko": FAR[1]}, ARG), ({"qo": FAR[4]}, ARG), ({"ko": FAR[4] - 8}, ARG),
        # q, k and v side by side in one buffer, turned where they are; then one column too far
        (dict(qo=FAR[0], k=FAR[0] + 512, ko=FAR[0] + 512, qs=(8 * 640, 640, 64), qos=(8 * 640, 640, 64), ks=(8 * 640, 640, 64),
              kos=(8 * 640, 640, 64)), fa.FA_OK),
        (dict(qo=FAR[0], k=FAR[0] + 510, ko=FAR[0] + 510, qs=(8 * 640, 640, 64), qos=(8 * 640, 640, 64), ks=(8 * 640, 640, 64),
              kos=(8 * 640, 640, 64)), ARG)])


def test_rotary_turns_travel_with_the_call(step):
    assert step.call("fa_rotary", rotary(r=32)) == fa.FA_OK
    assert [step.L.ss_turn(i) for i in (0, 15, 16)] == [1, 16, 0] and step.L.ss_copies()
    assert step.call("fa_rotary", rotary(r=32, qo=FAR[0], ko=FAR[2])) == fa.FA_OK and not step.L.ss_copies()


def test_group_norm(step):
    check(step, "fa_group_norm", norm, [
        ({"flags": 1}, ARG), ({"dtype": 9}, DTYPE), ({"param": 9}, DTYPE), ({"act": 4}, ARG), ({"act": -1}, ARG), ({"eps": -1e-9}, ARG),
        ({"eps": NAN}, ARG), ({"n": 1 << 31}, RANGE), ({"P": 1 << 31}, RANGE), ({"C": 0}, RANGE), ({"C": 8200, "G": 8}, RANGE),
        ({"G": 0}, RANGE), ({"G": 5}, RANGE), ({"x": None}, ARG), ({"y": None}, ARG), ({"x": FAR[0] + 1}, ARG), ({"gamma": FAR[2] + 2}, ARG),
        ({"gamma": None, "beta": None, "mean": None, "rstd": None}, fa.FA_OK), ({"n": 0, "x": None, "y": None}, fa.FA_OK),
        ({"P": 0, "x": None, "y": None}, fa.FA_OK), ({"ldx": HUGE}, RANGE), ({"ldy": 31}, RANGE), ({"sy": 99 * 32}, RANGE),
        ({"P": (1 << 31) - 1, "ldx": (1 << 40) - 1}, RANGE), ({"ldx": 0}, fa.FA_OK),
        ({"y": FAR[0]}, fa.FA_OK), ({"y": FAR[0], "ldx": 40}, ARG), ({"y": FAR[0] + 2}, ARG), ({"y": FAR[2]}, ARG), ({"mean": FAR[0]}, ARG),
        ({"rstd": FAR[4] + 4}, ARG), ({"mean": FAR[1] + 64}, ARG),
        ({"x": FAR[1] + 64, "ldx": 64, "ldy": 64}, fa.FA_OK), ({"x": FAR[1] + 62, "ldx": 64, "ldy": 64}, ARG)])


def test_group_norm_backward(step):
    check(step, "fa_group_norm_backward", norm_backward, [
        ({"flags": 1}, ARG), ({"dtype": 9}, DTYPE), ({"act": 7}, ARG), ({"G": 3}, RANGE), ({"x": None}, ARG), ({"dout": None}, ARG),
        ({"dx": None}, ARG), ({"mean": None}, ARG), ({"rstd": None}, ARG), ({"d_gamma": None, "d_beta": None}, fa.FA_OK),
        ({"n": 0, "x": None, "dout": None, "dx": None, "mean": None, "rstd": None}, fa.FA_OK),
        ({"P": 0, "x": None, "dout": None, "dx": None, "d_gamma": None, "d_beta": None}, fa.FA_OK),
        ({"dx": FAR[0]}, fa.FA_OK), ({"dx": FAR[1]}, fa.FA_OK), ({"dx": FAR[1], "ldd": 48}, ARG), ({"dx": FAR[0] + 2}, ARG),
        ({"dx": FAR[4]}, ARG), ({"d_gamma": FAR[2]}, ARG), ({"d_beta": FAR[7] + 4}, ARG), ({"d_beta": FAR[6]}, ARG), ({"lddx": 16}, RANGE)])


def test_orthogonalise(step):
    flat = dict(u=FAR[0], su=40000, out=FAR[0] + 2 * 6000, so=40000)       # two keys of one layer, layers 40000 apart
    check(step, "fa_orthogonalise", ortho, [
        ({"flags": 2}, ARG), ({"din": 9}, DTYPE), ({"dout": 9}, DTYPE), ({"mu": NAN}, ARG), ({"alpha": INF}, ARG), ({"beta": 1e31}, ARG),
        ({"eps": 0.0}, ARG), ({"eps": NAN}, ARG), ({"eps": 1e31}, ARG), ({"steps": 33}, RANGE), ({"rows": 1 << 24, "cols": 1}, RANGE),
        ({"rows": 40000, "cols": 40000}, RANGE), ({"rows": 1 << 20, "cols": 1 << 13}, RANGE), ({"count": 1 << 31}, RANGE),
        ({"abc": (3.0, 2.0, 1.0)}, RANGE), ({"abc": (5.0, 0.0, 0.0), "steps": 1}, RANGE), ({"abc": (5.0, 0.0, 0.0), "steps": 0}, fa.FA_OK),
        ({"abc": (NAN, 0.0, 0.0)}, ARG), ({"u": None}, ARG), ({"out": None}, ARG), ({"out": FAR[4] + 1}, ARG),
        ({"count": 0, "u": None, "out": None}, fa.FA_OK), ({"rows": 0, "u": None, "out": None}, fa.FA_OK), ({"ldu": HUGE}, RANGE),
        ({"ldo": 59}, RANGE), ({"so": 5999}, RANGE), ({"rows": 20, "so": 1199}, RANGE), ({"su": 0, "ldu": 0}, fa.FA_OK),
        ({"out": FAR[0]}, fa.FA_OK), ({"out": FAR[0], "dout": "f32"}, ARG), ({"out": FAR[0] + 2}, ARG), ({"out": FAR[0], "ldu": 61}, ARG),
        ({"res": FAR[4]}, fa.FA_OK), ({"res": FAR[4] + 2}, ARG), ({"res": FAR[4] + 2, "beta": 0.0}, fa.FA_OK),
        ({"m": FAR[2], "mo": FAR[2]}, fa.FA_OK), ({"m": FAR[2], "mo": FAR[2] + 4}, ARG), ({"m": FAR[2], "mo": FAR[3]}, fa.FA_OK),
        ({"mo": FAR[0]}, ARG), ({"mo": FAR[4]}, ARG), ({"m": FAR[4]}, ARG), ({"mo": FAR[2], "ldmo": 59}, RANGE),
        ({"mo": FAR[2] + 2}, ARG), (flat, fa.FA_OK), ({**flat, "out": FAR[0] + 2 * 5999}, ARG)])


def test_a_short_side_takes_one_launch_and_others_their_products(step):
    step.L.ss_reset(0)
    assert step.call("fa_orthogonalise", ortho(rows=16, cols=900)) == fa.FA_OK
    assert (step.L.ss_small(), step.L.ss_products(), step.L.ss_launches()) == (1, 0, 1)
    step.L.ss_reset(0)
    # square: three products a step
    assert step.call("fa_orthogonalise", ortho(rows=100, cols=100)) == fa.FA_OK
    assert step.L.ss_products() == 15
    step.L.ss_reset(0)
    # twice as wide, bf16: segments of three and two steps; fp32: the steps as they stand
    assert step.call("fa_orthogonalise", ortho(rows=100, cols=200)) == fa.FA_OK
    assert step.L.ss_products() == (1 + 9 + 1) + (1 + 5 + 1)
    step.L.ss_reset(0)
    assert step.call("fa_orthogonalise", ortho(rows=100, cols=200, dout="f32", out=FAR[6])) == fa.FA_OK
    assert step.L.ss_products() == 15


@pytest.mark.parametrize("name,make,at", [("fa_rotary", rotary, 1), ("fa_group_norm", norm, 1), ("fa_group_norm_backward", norm_backward, 2),
                                          ("fa_orthogonalise", ortho, 2)])
def test_the_next_call_waits_for_what_a_failed_one_had_queued(name, make, at):
    s = Step()
    s.L.ss_reset(at)
    assert s.call(name, make(), 1) == fa.FA_ERR_CUDA and "name" in s.error()
    assert "record:1" in s.log()
    s.L.ws_clear_log()
    assert s.call(name, make(), 2) == fa.FA_OK
    assert "wait:2" in s.log()
    assert s.close() == fa.FA_OK


def test_null_handles_and_arguments(step):
    for name in ("fa_rotary", "fa_group_norm", "fa_group_norm_backward", "fa_orthogonalise"):
        assert getattr(step.L, name)(None, None, None) == ARG
        assert getattr(step.L, name)(step.h, None, None) == ARG


def test_turns():
    """The frequencies against their formulas, in units of 2^-64 turns; and what is refused."""
    if not os.path.exists(fa.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()

    def near(turns, freq):
        assert len(turns) == len(freq)
        for t, f in zip(turns, freq):
            assert abs(t / 2 ** 64 - f / (2 * math.pi)) <= 1e-14 * f

    base = [10000.0 ** (-2 * i / 128) for i in range(64)]
    near(fa.rotary_turns(128), base)
    near(fa.rotary_turns(128, 10000.0, "linear", 4.0), [f / 4 for f in base])
    near(fa.rotary_turns(64, 10000.0, "base", 8.0), [(10000.0 * 8 ** (64 / 62)) ** (-2 * i / 64) for i in range(32)])
    near(fa.rotary_turns(2, 10000.0, "base", 8.0), [1.0])
    turns = [8192 * f / (2 * math.pi) for f in base]
    keep = [min(1.0, max(0.0, (t - 1) / 3)) for t in turns]
    near(fa.rotary_turns(128, 10000.0, "banded", 8.0, 8192.0, 1.0, 4.0), [f * (g + (1 - g) / 8) for f, g in zip(base, keep)])
    assert 0.0 in keep and 1.0 in keep
    for bad in ((3,), (0,), (514,), (64, 0.5), (64, math.inf), (64, 1e4, "linear", 0.5), (64, 1e4, "linear", NAN),
                (64, 1e4, "banded", 2.0, 0.0, 1.0, 4.0), (64, 1e4, "banded", 2.0, 8192.0, 4.0, 4.0), (64, 1e4, "banded", 2.0, 8192.0, -1.0, 4.0),
                (64, 1e300, "base", 1e300)):
        with pytest.raises(fa.FedAvgError):
            fa.rotary_turns(*bad)
    with pytest.raises(KeyError):
        fa.rotary_turns(64, 1e4, "other")


def test_positions_of_another_type_are_refused():
    import torch
    with pytest.raises(TypeError, match="int32"):
        fa.fa_rotary(None, 1, 4, 64, fa.rotary_turns(64), "f32", 1, 1, 2, position=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="layout"):
        fa.fa_rotary(None, 1, 4, 64, fa.rotary_turns(64), "f32", 1, 1, 2, layout="other")


def test_structs_have_the_headers_fields():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    ctype = {"uint32_t": ctypes.c_uint32, "int32_t": ctypes.c_int32, "uint64_t": ctypes.c_uint64, "int64_t": ctypes.c_int64,
             "double": ctypes.c_double, "fa_rotary_part": fa.fa_rotary_part}
    for name in ("fa_rotary_part", "fa_rotary_args", "fa_group_norm_args", "fa_group_norm_backward_args", "fa_orthogonalise_args"):
        body = re.search(r"typedef struct \{([^{}]*)\} " + name + r";", text).group(1)
        want = []
        for decl in filter(None, (d.strip() for d in body.split(";"))):
            pointer = "*" in decl
            kind, names = decl.replace("const ", "").replace("*", " ").split(None, 1)
            want += [(n.strip(), ctypes.c_void_p if pointer else ctype[kind]) for n in names.split(",")]
        assert list(getattr(fa, name)._fields_) == want, name


def test_an_output_in_place_has_its_inputs_strides_dimension_by_dimension(step):
    """Two dimensions of one extent whose strides are exchanged cover the same elements, each at
    another place: the kernels would write what they still have to read."""
    def taken(name, args):
        step.L.ss_reset(0)
        status = step.call(name, args)
        assert (status == fa.FA_OK) == (step.L.ss_launches() > 0), name
        return status

    one = dict(batch=1, seq=4, qh=4, kh=0, k=None, ko=None, qo=FAR[0], qs=(0, 256, 64))
    assert taken("fa_rotary", rotary(**one, qos=(0, 256, 64))) == fa.FA_OK
    assert taken("fa_rotary", rotary(**one, qos=(0, 64, 256))) == ARG
    batch = dict(batch=4, seq=4, qh=1, kh=0, k=None, ko=None, qo=FAR[0], qs=(256, 64, 64))
    assert taken("fa_rotary", rotary(**batch, qos=(256, 64, 999))) == fa.FA_OK            # a single head: its stride is not used
    assert taken("fa_rotary", rotary(**batch, qos=(64, 256, 64))) == ARG
    # only q is where it was: what does not turn is still copied for k
    assert taken("fa_rotary", rotary(r=32, qo=FAR[0])) == fa.FA_OK and step.L.ss_copies()
    square = dict(n=4, P=4, ldx=32, sx=128, y=FAR[0])
    assert taken("fa_group_norm", norm(**square, ldy=32, sy=128)) == fa.FA_OK
    assert taken("fa_group_norm", norm(**square, ldy=128, sy=32)) == ARG
    assert taken("fa_group_norm", norm(n=1, P=4, ldx=32, sx=128, y=FAR[0], ldy=32, sy=4096)) == fa.FA_OK    # a single sample
    for over in (FAR[0], FAR[1]):
        for lddx, step_dx, want in ((32, 128, fa.FA_OK), (128, 32, ARG)):
            args = norm_backward(n=4, P=4, dx=over, ldx=32, ldd=32, lddx=lddx)
            args.step_x = args.step_d = 128
            args.step_dx = step_dx
            assert taken("fa_group_norm_backward", args) == want
    many = dict(count=100, rows=100, ldu=60, su=6000, out=FAR[0])
    assert taken("fa_orthogonalise", ortho(**many, ldo=60, so=6000)) == fa.FA_OK
    assert taken("fa_orthogonalise", ortho(**many, ldo=6000, so=60)) == ARG
    far = dict(count=100, rows=100, ldm=60, sm=6000, m=FAR[2], mo=FAR[2])
    assert taken("fa_orthogonalise", ortho(**far, ldmo=60, smo=6000)) == fa.FA_OK
    assert taken("fa_orthogonalise", ortho(**far, ldmo=6000, smo=60)) == ARG
    weight = dict(count=100, rows=100, res=FAR[4], ldr=60, sr=6000)
    assert taken("fa_orthogonalise", ortho(**weight, ldo=60, so=6000)) == fa.FA_OK
    assert taken("fa_orthogonalise", ortho(**weight, ldo=6000, so=60)) == ARG
