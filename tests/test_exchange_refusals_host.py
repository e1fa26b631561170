"""Refusals of the gradient of the expert combine: no GPU, nothing launched."""

import pytest

from chunk_schedule_execution_amd import capi

P = 1 << 20  # an aligned address that no refused call looks at
ARGS = ("dout", "h", "positions", "slots", "gates", "dh", "dgates")


def call(**kw):
    a = dict(dict.fromkeys(ARGS, P), **kw)
    capi.ccl_expert_combine_backward(capi.CCL_F32, a["dout"], 0, a["h"], 0, a["positions"], a["slots"], a["gates"], 8, 2,
                                     64, a["dh"], 0, a["dgates"])


# what a call with these outputs reads
READ = {"both": ("dout", "h", "positions", "slots"), "dh": ("dout", "positions", "slots"),
        "dgates": ("dout", "h", "positions", "slots")}


@pytest.mark.parametrize("outputs,name", [(o, n) for o in READ for n in READ[o]])
def test_a_null_operand_is_refused(outputs, name):
    kw = {"both": {}, "dh": dict(dgates=0), "dgates": dict(dh=0)}[outputs]
    with pytest.raises(capi.CCLError) as e:
        call(**kw, **{name: 0})
    assert e.value.status == capi.CCL_ERR_INVALID_ARGUMENT and name in capi.ccl_last_error_detail()


@pytest.mark.parametrize("outputs,name", [(o, n) for o in READ for n in READ[o] + ("gates",)] +
                         [("both", "dh"), ("both", "dgates"), ("dh", "dh"), ("dgates", "dgates")])
def test_a_misaligned_operand_is_refused(outputs, name):
    kw = {"both": {}, "dh": dict(dgates=0), "dgates": dict(dh=0)}[outputs]
    with pytest.raises(capi.CCLError) as e:
        call(**dict(kw, **{name: P + 2}))
    assert e.value.status == capi.CCL_ERR_INVALID_ARGUMENT and name in capi.ccl_last_error_detail()
