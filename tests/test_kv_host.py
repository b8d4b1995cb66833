"""Host checks of the decode-state sources and binding (no GPU)."""
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantised_weight_gb300", "csrc")


def test_prompt_kernel_waits_for_stored_probabilities():
    """Stores to tensor memory are asynchronous, and nothing orders a load of the same columns behind
    them but a wait for the stores: the first half's probabilities are read back only after one."""
    src = open(os.path.join(CSRC, "kv_prompt.cu")).read()
    at = src.index("if (half == 1) {")
    calls = re.findall(r"\b(tmem_stored|tmem_load32|tmem_store32)\(", src[at:])
    assert calls[:3] == ["tmem_stored", "tmem_load32", "tmem_store32"]
