"""`profiling case` names the listed cases when asked for another (CPU only)."""
import pytest

from gguf_block_quant_qmm_amd import profiling
from perf import operators


def test_an_unknown_case_is_refused_with_the_names():
    with pytest.raises(SystemExit) as e:
        profiling.main(["case", "--name", "nothing"])
    assert all(c["name"] in str(e.value) for c in operators.listed()) and operators.own is False
