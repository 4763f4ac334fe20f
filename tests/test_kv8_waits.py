"""The tcgen05 kernel's bounded waits, as the source has them: a wait that runs out is
voted on by the whole CTA before anything that products may still use is touched, and the
CTA waits once more before it frees its tensor memory."""
import pathlib
import re

SRC = pathlib.Path(__file__).resolve().parent.parent / "paged_kv_decode_16_gb300" / "csrc"


def test_every_wait_is_voted_on():
    text = re.sub(r"//[^\n]*", "", (SRC / "kv8_umma.cu").read_text())
    text = re.sub(r"\s+", " ", text)
    voted = text.count("__syncthreads_or(!mbar_wait_bounded(")
    last = re.findall(r"if \(fail\) \{ flags \|= PKV_DEV_TIMEOUT; mbar_wait_bounded\(bar, ph\); \}",
                      text)
    assert len(last) == 1
    assert text.count("mbar_wait_bounded(") == voted + 1
    # each call of the voted wait leaves the loop when it gave up
    calls = text.count("fail = wait_all();")
    assert calls >= 3 and text.count("fail = wait_all(); if (fail) break;") == calls
    # nothing frees tensor memory before that last wait
    assert text.index("tmem_dealloc(tmem") > text.index("mbar_wait_bounded(bar, ph); }")
