"""Sizes next to what 32-bit column arithmetic holds are refused on the host (no GPU)."""
import pytest

import chunked_lm_head_tcgen05_gb300 as lm
from test_operators_host import (LOGITS_BWD, LOGITS_FWD, PROCESS_BWD, PROCESS_FWD, UNSUPPORTED, call)

CASES = [("lmhead_distill_logits_fwd", LOGITS_FWD), ("lmhead_distill_logits_bwd", LOGITS_BWD),
         ("lmhead_process_logits_fwd", PROCESS_FWD), ("lmhead_process_logits_bwd", PROCESS_BWD)]


@pytest.mark.parametrize("name,defaults", CASES)
@pytest.mark.parametrize("V", [2 ** 31 - 1, 2 ** 31 - 1024])
def test_vocabulary(name, defaults, V):
    lm.build()
    wide = {k: V for k in ("ld", "out_ld", "d_ld", "grad_ld") if k in defaults}
    assert call(getattr(lm.library(), name), defaults, V=V, **wide) == UNSUPPORTED
