"""Host checks of the sources of the attention over a shared prefix (no GPU): what a wait that gave up must not lead to."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_quantised_weight_gb300", "csrc")


def source(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_no_wait_is_without_a_limit_or_a_verdict():
    """Waits end by themselves, and what they say reaches the warp's own flag, but for those of the copies in flight,
    behind which nothing comes."""
    src = source("kv_prefix.cuh")
    assert not re.search(r"while\s*\(\s*!\s*(__all_sync\(~0u,\s*)?mbar_try_wait", src)
    for m in re.finditer(r"[^;{}]*\bmbar_wait_bounded\([^;]*;", src):
        assert re.search(r"return|\(void\)", m.group()), m.group()
    for m in re.finditer(r"[^;{}]*\bwait_on\([^;{]*[;{]", src):
        assert re.search(r"dead =|bool wait_on", m.group()), m.group()


def test_nothing_is_expected_by_a_warp_that_gave_up():
    """Bytes are announced once a slot is known to be free, and a slot goes back only once its bytes have landed: a barrier
    never counts the bytes of two copies."""
    src = source("kv_prefix.cuh")
    for m in re.finditer(r"mbar_arrive_expect_tx", src):
        assert "if (dead) return;" in src[m.start() - 200:m.start()]
    back = re.findall(r"([^\n]*)arrive_on\([kv]raw_empty", src)
    assert len(back) == 2 and all("!dead" in line for line in back)
    issues = re.findall(r"if \(([^\n]*)elect_one\(\)", src)
    assert len(issues) == 2 and all(cond == "!dead && " for cond in issues)


def test_a_ring_holds_a_whole_step():
    """A converter waits for the scales, which come behind all copies of a step: fewer slots than a step's tiles would wait
    for one another."""
    src = source("kv_prefix.cuh")
    assert "static_assert(kRawV >= RT && kRawK >= RT" in src
    copies, scales = src.index("mbar_arrive_expect_tx"), src.index("arrive_on(sc_full")
    assert copies < scales


def test_copies_in_flight_are_waited_for():
    """Shared memory is theirs until they land, in a warp that gave up too."""
    src = source("kv_prefix.cuh")
    at = src.index("if (dead) {")
    for ring in ("kraw_full", "vraw_full"):
        assert f"(void)mbar_wait_bounded({ring}" in src[at:at + 900]


def test_the_checks_above_find_what_they_check():
    """Each of the searches above meets the sources' calls: a renamed helper is not passed over."""
    src = source("kv_prefix.cuh")
    assert len(re.findall(r"[^;{}]*\bmbar_wait_bounded\([^;]*;", src)) == 3
    assert len(re.findall(r"[^;{}]*\bwait_on\([^;{]*[;{]", src)) == 2
    assert src.count("mbar_arrive_expect_tx") == 1
    assert src.count("mbar_try_wait") == 2  # tried once each: in wait() and ahead of a step
