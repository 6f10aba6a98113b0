"""Results over a call's own input need that input's layout: with rows another distance apart, or of
another type, one row's result would overwrite another row's input before it is read.  Such calls
are refused on the host (no GPU)."""
import pytest

import chunked_lm_head_tcgen05_gb300 as lm
from test_operators_host import (INVALID, LOGITS_BWD, NORM_BWD, NORM_FWD, PROCESS_BWD, PROCESS_FWD, P,
                                 call)

A, B, C = P(1 << 20), P(1 << 24), P(1 << 28)

CASES = [
    ("lmhead_process_logits_fwd", PROCESS_FWD, dict(logits=A, out=A, ld=100, out_ld=104)),
    ("lmhead_process_logits_bwd", PROCESS_BWD, dict(grad=A, d=A, logits=B, grad_ld=104, d_ld=100)),
    ("lmhead_process_logits_bwd", PROCESS_BWD, dict(grad=A, d=B, logits=B, ld=104, d_ld=100)),
    ("lmhead_distill_logits_bwd", LOGITS_BWD, dict(logits=A, d=A, ld=100, d_ld=128)),
    ("lmhead_layernorm_fwd", NORM_FWD, dict(x=A, y=A, x_ld=64, y_ld=72)),
    ("lmhead_layernorm_fwd", NORM_FWD, dict(x=A, y=A, x_type=0, y_type=1, param_type=0)),
    ("lmhead_layernorm_bwd", NORM_BWD, dict(dy=A, dx=A, x=B, dy_type=1, dy_ld=72, workspace=C)),
    ("lmhead_layernorm_bwd", NORM_BWD, dict(dy=A, dx=A, x=B, dy_type=0, workspace=C)),
    ("lmhead_layernorm_bwd", NORM_BWD, dict(dy=A, dx=B, x=B, x_ld=72, workspace=C)),
]


@pytest.mark.parametrize("name,defaults,over", CASES)
def test_over_an_input_of_another_layout(name, defaults, over):
    lm.build()
    assert call(getattr(lm.library(), name), defaults, **over) == INVALID
