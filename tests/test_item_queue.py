"""The marks that go with the packed prefill's work items (item_queue.cuh, compiled for the host): over every
interleaving of publisher, marking warps and reading warps, a reader sees exactly its own item's mark."""
import os
import subprocess
import tempfile

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "mixed_head_kv_b200", "csrc")


def test_a_reader_sees_its_own_items_mark():
    with tempfile.TemporaryDirectory() as d:
        exe = os.path.join(d, "item_queue_check")
        subprocess.check_call(["g++", "-O1", "-std=c++17", "-I", CSRC, os.path.join(HERE, "item_queue_check.cpp"), "-o", exe])
        out = dict((line.split()[0], line.split()[1:]) for line in subprocess.check_output([exe], text=True).splitlines())
    states, wrong = map(int, out["marks"])
    assert states > 10000 and wrong == 0
    # Clearing the place of four items ago is not enough: a reader frees a slot when it takes the item.
    assert int(out["clears"][1]) > 0


def test_the_kernel_uses_these_marks():
    text = open(os.path.join(CSRC, "prefill_packed.cu")).read()
    assert text.count("marked_odd[mark_place(ord)]") == 2 and "odd_values[" not in text
