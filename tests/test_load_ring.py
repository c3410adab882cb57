"""The loaders' ring (csrc/load_ring.cuh) on the host, against modelled barriers."""
import os
import re
import shutil
import subprocess

import pytest

from test_sources import CSRC, _code

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def build(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host compiler")

    def make(*flags):
        exe = str(tmp_path_factory.mktemp("ring") / "ring")
        subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-I", CSRC, *flags,
                        os.path.join(HERE, "load_ring.cpp"), "-o", exe], check=True)
        return subprocess.run([exe], capture_output=True, text=True, timeout=120)
    return make


def test_no_copy_follows_a_wait_that_gave_up(build):
    p = build()
    assert p.returncode == 0, p.stdout


def test_the_model_shows_a_loader_that_copies_on(build):
    p = build("-DCARRY_ON")
    assert p.returncode == 1, (p.returncode, p.stdout)


@pytest.mark.parametrize("name", ["dense_decode.cu", "decode.cu", "index_score_tc.cu",
                                  "prefill_index.cu"])
def test_loaders_look_at_what_their_waits_say(name):
    """A wait for a stage to be free is never a statement of its own (one for an
    accumulator may be: no copies go there)."""
    text = _code(os.path.join(CSRC, name))
    assert re.search(r"\bLoadRing<", text)
    assert not re.search(r"(^|[;{})])\s*mbar_wait\(&(?:\w+\.)*(?!acc_)\w*empty", text)


def _statements(name, barrier):
    """Waits for a barrier whose answer is dropped."""
    return re.findall(r"(?:^|[;{})])\s*mbar_wait\(&%s\b" % barrier, _code(os.path.join(CSRC, name)))


@pytest.mark.parametrize("name,barrier", [("decode.cu", b) for b in
                                          ("item_full", "meta_full", "item_empty")]
                         + [("index_score_tc.cu", "full")])
def test_records_are_read_after_a_wait_that_succeeded_only(name, barrier):
    """A record that was not published holds any bytes: pages and rows of them would be
    addresses outside every buffer, and warps that read different ones would wait for
    each other in different barriers."""
    text = _code(os.path.join(CSRC, name))
    assert re.search(r"mbar_wait\(&%s\b" % barrier, text)
    assert not _statements(name, barrier)


def test_the_prefills_issuer_loads_nothing_after_a_wait_that_gave_up():
    """Its loads are single: each of their functions asks whether a wait gave up, and
    every wait of the issuer answers."""
    text = _code(os.path.join(CSRC, "prefill.cu"))
    for barrier in ("k_full", "k_free", "vt_ready"):
        assert re.search(r"mbar_wait\(&%s\b" % barrier, text)
        assert not _statements("prefill.cu", barrier), barrier
    loads = re.findall(r"\bauto load_\w+ = \[&\]\([^)]*\) \{(.*?)\n  \};", text, flags=re.S)
    assert len(loads) == 3
    for body in loads:
        assert "if (!going) return;" in body[:body.index("mbar_arrive_expect_tx")]
    # a buffer of queries is armed again once its last copies are there, come what may
    assert re.search(r"!mbar_wait\(&s_ready\[w\][^;]*?\)\)\s*mbar_drain\(&q_full\[w\]", text)


@pytest.mark.parametrize("name", ["decode.cu", "dense_decode.cu", "index_score_tc.cu",
                                  "prefill_index.cu", "prefill.cu", "tree_attention.cu"])
def test_what_a_block_issued_ends_before_it_retires(name):
    """A loader or MMA warp that looks for a timeout before the block's other warps are
    done can miss one that they meet later: it waits for what it issued in any case, or
    looks after a barrier with them."""
    text = _code(os.path.join(CSRC, name))
    assert not re.search(r"&\s*MSA_DEVERR_TIMEOUT", text)
    drains = [m.start() for m in re.finditer(r"\bmbar_drain\(", text)]
    assert drains
    for m in re.finditer(r"\btimed_out\(", text):
        before, after = text[max(0, m.start() - 250):m.start()], text[m.start():m.start() + 150]
        if "mbar_drain(" in after:
            assert re.search(r"__syncthreads\(\);|named_bar_sync\(kDone,", before), before
