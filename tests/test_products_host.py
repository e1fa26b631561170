"""Refusals and workspace queries of the products and the row exchange: no GPU, nothing
launched. Every refused call names an error before any device work."""

import pytest
import torch

from chunk_schedule_execution_amd import capi, ops
from oracle import products as O

P = 1 << 20  # an aligned address that no refused call looks at


def desc(**kw):
    d = dict(dtype=capi.CCL_BF16, activation=capi.CCL_ACT_SILU, rows=8, in_features=16, out_features=24)
    d.update(kw)
    return capi.ccl_linear_desc(**d)


BAD_DESC = [
    (dict(dtype=capi.CCL_I32), capi.CCL_ERR_UNSUPPORTED),
    (dict(dtype=9), capi.CCL_ERR_UNSUPPORTED),
    (dict(activation=-1), capi.CCL_ERR_UNSUPPORTED),
    (dict(activation=5), capi.CCL_ERR_UNSUPPORTED),
    (dict(rows=-1), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(rows=1 << 31), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(in_features=0), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(in_features=(1 << 20) + 1), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(out_features=0), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_x=15), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_w=15), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_out=23), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_residual=-24), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_preact=(1 << 22) + 1), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_dx=1), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(ld_dw=1), capi.CCL_ERR_INVALID_ARGUMENT),
    (dict(flags=2), capi.CCL_ERR_INVALID_ARGUMENT),
]


def refused(status, f, *args):
    with pytest.raises(capi.CCLError) as e:
        f(*args)
    assert e.value.status == status and capi.ccl_last_error_detail()


@pytest.mark.parametrize("bad,status", BAD_DESC + [(dict(experts=2), capi.CCL_ERR_INVALID_ARGUMENT)])
def test_linear_refuses_bad_descriptors(bad, status):
    d = desc(**bad)
    refused(status, capi.ccl_linear_workspace, d, False, False)
    refused(status, capi.ccl_linear, d, P, P, 0, 0, P, 0, P, 1 << 40)
    refused(status, capi.ccl_linear_backward, d, P, P, P, P, P, P, P, P, 1 << 40)


@pytest.mark.parametrize("bad,status", BAD_DESC + [(dict(experts=0), capi.CCL_ERR_INVALID_ARGUMENT),
                                                   (dict(experts=4097), capi.CCL_ERR_INVALID_ARGUMENT)])
def test_grouped_linear_refuses_bad_descriptors(bad, status):
    d = desc(**dict(dict(experts=4), **bad))
    refused(status, capi.ccl_linear_workspace, d, True, False)
    refused(status, capi.ccl_grouped_linear, d, P, P, P, 0, P, 0, P, 1 << 40)
    refused(status, capi.ccl_grouped_linear_backward, d, P, P, P, P, P, P, P, P, P, 1 << 40)


def test_null_descriptor():
    lib = capi.lib()
    assert lib.ccl_linear(None, P, P, 0, 0, P, 0, 0, 0, 0) == capi.CCL_ERR_INVALID_ARGUMENT
    assert lib.ccl_linear_workspace(None, 0, 0) == capi.CCL_ERR_INVALID_ARGUMENT


FORWARD = ["x", "w", "bias", "residual", "out", "preact"]


@pytest.mark.parametrize("name", ["x", "w", "out"])
def test_linear_refuses_null_operands(name):
    args = dict.fromkeys(FORWARD, P)
    args[name] = 0
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_linear, desc(), *args.values(), P, 1 << 40)


@pytest.mark.parametrize("name", FORWARD)
def test_linear_refuses_misaligned_operands(name):
    args = dict.fromkeys(FORWARD, P)
    args[name] = P + 2  # an element's alignment: refused unless the descriptor says so
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_linear, desc(), *args.values(), P, 1 << 40)
    args[name] = P + 1  # not even an element's
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_linear, desc(flags=capi.CCL_LINEAR_UNALIGNED), *args.values(), P,
            1 << 40)


BACKWARD = ["dout", "x", "w", "preact", "dx", "dw", "dbias"]


@pytest.mark.parametrize("name", ["dout", "x", "w", "preact"])
def test_linear_backward_refuses_null_operands(name):
    args = dict.fromkeys(BACKWARD, P)
    args[name] = 0
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_linear_backward, desc(), *args.values(), P, 1 << 40)


@pytest.mark.parametrize("name", BACKWARD)
def test_linear_backward_refuses_misaligned_operands(name):
    args = dict.fromkeys(BACKWARD, P)
    args[name] = P + 2
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_linear_backward, desc(), *args.values(), P, 1 << 40)


def test_grouped_refuses_null_and_misaligned_offsets():
    for o in (0, P + 2):
        refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_grouped_linear, desc(experts=3), o, P, P, 0, P, 0, P, 1 << 40)
        refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_grouped_linear_backward, desc(experts=3), o, P, P, P, P, P, P,
                P, P, 1 << 40)


def test_workspace_is_checked():
    d = desc()
    need = capi.ccl_linear_workspace(d, False, True)
    assert need > 0
    args = dict.fromkeys(BACKWARD, P)
    for ws, have in ((0, need), (P, need - 1), (P + 8, need)):
        refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_linear_backward, d, *args.values(), ws, have)


@pytest.mark.parametrize("dtype", [capi.CCL_F32, capi.CCL_BF16])
@pytest.mark.parametrize("experts", [0, 1, 64, 4096])
@pytest.mark.parametrize("rows", [0, 1, 17, 1000, 2**31 - 1])
def test_workspace_of_every_size(rows, experts, dtype):
    for k, n in ((1, 1), (8, 8), (33, 1 << 20), (1 << 20, 33), (4096, 4096)):
        for backward in (False, True):
            d = desc(dtype=dtype, rows=rows, in_features=k, out_features=n, experts=experts)
            assert capi.ccl_linear_workspace(d, experts > 0, backward) >= 0


def test_workspace_grows_with_the_rows():
    last = -1
    for rows in (0, 1, 100, 10000, 1 << 20):
        need = capi.ccl_linear_workspace(desc(rows=rows, experts=5), True, True)
        assert need >= last
        last = need


def test_forward_of_no_rows_is_done_at_once():
    capi.ccl_linear(desc(rows=0), 0, 0, 0, 0, 0, 0, 0, 0)


@pytest.mark.parametrize("tokens,choices,experts", [(-1, 1, 1), (1, 0, 1), (1, 1025, 1), (1, 1, 0), (1, 1, 1025),
                                                    (1 << 30, 2, 4)])
def test_route_refuses_bad_sizes(tokens, choices, experts):
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_expert_route_workspace, tokens, choices, experts)
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_expert_route, P, tokens, choices, experts, P, P, P, P, 1 << 40)


def test_route_refuses_bad_pointers():
    need = capi.ccl_expert_route_workspace(100000, 2, 8)
    for i in range(4):
        for bad in (0, P + 2):
            p = [P] * 4
            p[i] = bad
            refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_expert_route, p[0], 100000, 2, 8, p[1], p[2], p[3], P,
                    need)
    refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_expert_route, P, 100000, 2, 8, P, P, P, P, need - 1)


@pytest.mark.parametrize("bad", [dict(dtype=capi.CCL_I32), dict(tokens=-1), dict(choices=0), dict(width=0),
                                 dict(width=(1 << 20) + 1), dict(ld=63), dict(tokens=1 << 31)])
def test_exchange_refuses_bad_sizes(bad):
    a = dict(dtype=capi.CCL_F32, tokens=8, choices=2, width=64, ld=0)
    a.update(bad)
    status = capi.CCL_ERR_UNSUPPORTED if "dtype" in bad else capi.CCL_ERR_INVALID_ARGUMENT
    t, c, w, ld = a["tokens"], a["choices"], a["width"], a["ld"]
    refused(status, capi.ccl_expert_dispatch, a["dtype"], P, ld, P, t, c, w, P, 0)
    refused(status, capi.ccl_expert_combine, a["dtype"], P, ld, P, P, t, c, w, P, 0)
    refused(status, capi.ccl_expert_combine_backward, a["dtype"], P, ld, P, 0, P, P, P, t, c, w, P, 0, P)


def test_exchange_refuses_bad_pointers():
    for bad in (0, P + 2):
        for i in range(3):
            p = [P] * 3
            p[i] = bad
            refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_expert_dispatch, capi.CCL_F32, p[0], 0, p[1], 8, 2, 64,
                    p[2], 0)
            refused(capi.CCL_ERR_INVALID_ARGUMENT, capi.ccl_expert_combine, capi.CCL_F32, p[0], 0, p[1], 0, 8, 2, 64,
                    p[2], 0)


def test_wrappers_refuse_host_tensors_and_wrong_shapes():
    x, w = torch.zeros(4, 8), torch.zeros(6, 8)
    with pytest.raises(ValueError, match="GPU memory"):
        ops.linear(x, w)
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        ops.linear(x.half(), w.half())
    with pytest.raises(ValueError, match="matrix"):
        ops.linear(x[0], w)
    with pytest.raises(ValueError, match="GPU memory"):
        ops.expert_dispatch(x, torch.zeros(8, dtype=torch.int32), 2)
    with pytest.raises(ValueError, match="int32"):
        ops.expert_route(torch.zeros(4, 2), 8)
    with pytest.raises(ValueError, match="contiguous"):
        ops._ld(torch.zeros(8, 4).t(), "x")
    with pytest.raises(ValueError, match="overlap"):
        ops._ld(torch.zeros(1, 8).expand(4, 8), "x")
    with pytest.raises(ValueError, match="follow"):
        ops._ld(torch.zeros(3, 5, 8)[:, :4], "w")
    assert ops._ld(torch.zeros(4, 10)[:, :8], "x") == 10 and ops._ld(torch.zeros(3, 4, 8), "w") == 8


def test_oracle_slopes_against_differences():
    z = torch.linspace(-6, 6, 2001, dtype=torch.float64)
    for name in ("none", "gelu", "gelu_tanh", "silu"):
        d = (O.act(z + 1e-5, name) - O.act(z - 1e-5, name)) / 2e-5
        assert float((d - O.slope(z, name)).abs().max()) < 1e-8
        assert float(O.slope(z, name).abs().max()) <= O.STEEPEST


def test_oracle_route_by_hand():
    # choices of three tokens over experts 0..2; -1 and 7 are served elsewhere
    offsets, positions, slots = O.route([[2, 0], [-1, 2], [0, 7]], 3)
    assert offsets == [0, 2, 2, 4] and positions == [2, 0, -1, 3, 1, -1] and slots == [1, 4, 0, 3, -1, -1]
